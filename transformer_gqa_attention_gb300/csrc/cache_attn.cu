// cache_attn.cu — attention of a few positions per sequence over caches whose lengths differ
// from sequence to sequence: a tree of drafted tokens (each row sees the prefix and its own
// ancestors), and a decode step that adds each key's weight to a running sum.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "launch.h"
#include "ptx.cuh"

namespace gqa {

// One CTA per (position, kv group, sequence), one warp per query head; lane i holds elements
// 4i .. 4i+3 of the head.  Online softmax, one key at a time.
__global__ void __launch_bounds__(128) cache_attn_kernel(const CacheAttnParams p) {
  __shared__ float pw[4][32];
  griddep_wait();
  const int t = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int h = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = p.kv_len[b];
  const size_t row = (static_cast<size_t>(b) * p.T + t) * (p.n_kv * 512) + (g * 4 + h) * 128 + 4 * lane;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.h) + row;
  if (len < 0 || len > p.S_max - p.n_new) {
    if (threadIdx.x == 0) atomicOr(p.status, kDevErrRange);
    *reinterpret_cast<uint2*>(out) = make_uint2(0x7FC07FC0u, 0x7FC07FC0u);
    return;
  }
  const int W = (p.T + 31) / 32;
  const uint32_t* mask = p.mask ? p.mask + (static_cast<size_t>(b) * p.T + t) * W : nullptr;
  const uint2 qw = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.q) + row);
  const float q[4] = {bf16lo_to_f32(qw.x), bf16hi_to_f32(qw.x), bf16lo_to_f32(qw.y), bf16hi_to_f32(qw.y)};
  const size_t kv_row = static_cast<size_t>(p.n_kv) * 128;
  const size_t kv0 = (static_cast<size_t>(b) * p.S_max * p.n_kv + g) * 128 + 4 * lane;
  auto score = [&](int s) {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.k) + kv0 + s * kv_row);
    float d = q[0] * bf16lo_to_f32(w.x) + q[1] * bf16hi_to_f32(w.x) + q[2] * bf16lo_to_f32(w.y) +
              q[3] * bf16hi_to_f32(w.y);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    return d * p.scale_log2;
  };
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  const int end = len + p.n_new;
  for (int s = 0; s < end; ++s) {
    const int j = s - len;
    if (j >= 0 && mask && !((mask[j >> 5] >> (j & 31)) & 1u)) continue;
    const float x = score(s);
    const float m_new = fmaxf(m, x);
    const float a = m == -INFINITY ? 0.f : exp2f(m - m_new);
    const float e = m_new == -INFINITY ? 0.f : exp2f(x - m_new);
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.v) + kv0 + s * kv_row);
    l = l * a + e;
    acc[0] = acc[0] * a + e * bf16lo_to_f32(w.x);
    acc[1] = acc[1] * a + e * bf16hi_to_f32(w.x);
    acc[2] = acc[2] * a + e * bf16lo_to_f32(w.y);
    acc[3] = acc[3] * a + e * bf16hi_to_f32(w.y);
    m = m_new;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint2*>(out) =
      make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
  if (!p.weights) return;
  float* wsum = p.weights + (static_cast<size_t>(b) * p.n_kv + g) * p.S_max;
  for (int s0 = 0; s0 < end; s0 += 32) {
    for (int i = 0; i < min(32, end - s0); ++i) {
      const float e = exp2f(score(s0 + i) - m) * inv;
      if (lane == 0) pw[h][i] = e;
    }
    __syncthreads();
    if (h == 0 && s0 + lane < end) wsum[s0 + lane] += (pw[0][lane] + pw[1][lane]) + (pw[2][lane] + pw[3][lane]);
    __syncthreads();
  }
}

cudaError_t launch_cache_attn(const CacheAttnParams& p, cudaStream_t s) {
  return launch_pdl(cache_attn_kernel, dim3(p.T, p.n_kv, p.B), dim3(128), 0, s, 0, p);
}

}  // namespace gqa
