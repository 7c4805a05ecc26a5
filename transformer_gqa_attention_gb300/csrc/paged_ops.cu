// paged_ops.cu — rotation of queries by position, the table of a rotation, and the append of new keys
// and values to their pages.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "launch.h"
#include "rope.cuh"

namespace gqa {

namespace {
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ uint4 ld16(const void* p) { return ld_behind_wait(static_cast<const uint4*>(p)); }
}  // namespace

// ------------------------------------------------------------------------------ rotation
// grid (ceil(n_tok / kWarps), groups of heads_each heads); a warp per token and group: eight threads
// per head, four heads at a time, whose angles are the same.
__global__ void __launch_bounds__(kThreads) rope_apply_kernel(const __grid_constant__ RopeParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= p.n_tok) return;
  const int i = threadIdx.x & 7, sub = (threadIdx.x & 31) >> 3;
  const RopeLane at(p.rope, true, i);
  float2 cs[8];
  rope_coefficients(p.rope, at, i, __ldcg(p.positions + t), cs);
  const int h1 = min(p.n_heads, static_cast<int>(blockIdx.y + 1) * p.heads_each);
  for (int h = blockIdx.y * p.heads_each + sub; h < h1; h += 4) {
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + t * p.stride + h * 128;
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.out) + t * p.out_stride + h * 128;
    uint4 va = ld16(x + 8 * at.a), vb = ld16(x + 8 * at.b);
    if (at.turns) {
      float a[8], b[8];
      unpack8(va, a);
      unpack8(vb, b);
      rope_turn(p.rope.layout, cs, a, b);
      va = pack8(a);
      vb = pack8(b);
    }
    *reinterpret_cast<uint4*>(y + 8 * at.a) = va;
    *reinterpret_cast<uint4*>(y + 8 * at.b) = vb;
  }
}

cudaError_t launch_rope_apply(const RopeParams& p, cudaStream_t s) {
  const dim3 grid((p.n_tok + kWarps - 1) / kWarps, (p.n_heads + p.heads_each - 1) / p.heads_each);
  return launch_pdl(rope_apply_kernel, grid, dim3(kThreads), 0, s, 0, p);
}

// A thread per (token, pair).
__global__ void __launch_bounds__(kThreads) rope_table_kernel(const __grid_constant__ RopeParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int at = blockIdx.x * kThreads + threadIdx.x;
  const int t = at >> 6, j = at & 63;
  if (t >= p.n_tok) return;
  const float2 cs = 2 * j < p.rope.rot_dim ? rope_cos_sin(p.rope, j, __ldcg(p.positions + t)) : make_float2(1.f, 0.f);
  static_cast<float2*>(p.out)[at] = cs;
}

cudaError_t launch_rope_table(const RopeParams& p, cudaStream_t s) {
  return launch_pdl(rope_table_kernel, dim3((p.n_tok * 64 + kThreads - 1) / kThreads), dim3(kThreads), 0, s, 0, p);
}

// ------------------------------------------------------------------------------ append
// Eight values in the pools' type, divided by the scale (inv: its reciprocal).
__device__ __forceinline__ void store8(__nv_bfloat16* at, const float (&x)[8], float) {
  *reinterpret_cast<uint4*>(at) = pack8(x);
}
__device__ __forceinline__ void store8(uint8_t* at, const float (&x)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i] * inv, x[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi =
        __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2] * inv, x[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | hi << 16;
  }
  *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
}

// Eight threads per (token, head), as the rotation; hl heads (1, 2 or 4: what of n_kv fits) at a time,
// so that a warp holds 4 / hl tokens.
template <typename E>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const __grid_constant__ PagedAppendParams p, int hl) {
  griddep_launch_dependents();
  griddep_wait();
  const int group = (blockIdx.x * kThreads + threadIdx.x) >> 3;  // of eight threads
  const int i = threadIdx.x & 7;
  const int tok = group / hl, g0 = group - tok * hl;
  if (tok >= p.B * p.T) return;
  const int b = tok / p.T, t = tok - b * p.T;
  const int n = p.n_new ? __ldcg(p.n_new + b) : p.T;
  const int len = __ldcg(p.kv_len + b);
  if (n < 0 || n > p.T || len < 0 || len > p.max_pages * p.pool.page_size - n) {
    if (t == 0 && g0 == 0 && i == 0) atomicOr(p.status, kDevErrRange);
    return;
  }
  if (t >= n) return;
  const int s = len + t;
  const int in_table = s / p.pool.page_size;
  const int page = __ldcg(p.page_table + static_cast<size_t>(b) * p.max_pages + in_table);
  if (page < 0 || page >= p.pool.n_pages) {
    if (g0 == 0 && i == 0) atomicOr(p.status, kDevErrRange);
    return;
  }
  const RopeLane at(p.rope, p.rotate, i);
  float2 cs[8];
  rope_coefficients(p.rope, at, i, p.rope_pos ? __ldcg(p.rope_pos + b) + t : s, cs);
  const long long row = page * p.pool.page + (s - in_table * p.pool.page_size) * p.pool.pos;
  for (int g = g0; g < p.n_kv; g += hl) {
    const long long src = b * p.stride_b + t * p.stride_t + g * 128;
    const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.k) + src;
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v) + src;
    const uint4 ka = ld16(k + 8 * at.a), kb = ld16(k + 8 * at.b), va = ld16(v + 8 * at.a), vb = ld16(v + 8 * at.b);
    const float ik = p.pool.k_scale ? 1.f / __ldcg(p.pool.k_scale + g) : 1.f;
    const float iv = p.pool.v_scale ? 1.f / __ldcg(p.pool.v_scale + g) : 1.f;
    E* dk = static_cast<E*>(p.pool.k) + row + g * p.pool.head;
    E* dv = static_cast<E*>(p.pool.v) + row + g * p.pool.head;
    float x[8], y[8];
    unpack8(ka, x);
    unpack8(kb, y);
    if (at.turns) rope_turn(p.rope.layout, cs, x, y);
    store8(dk + 8 * at.a, x, ik);
    store8(dk + 8 * at.b, y, ik);
    unpack8(va, x);
    unpack8(vb, y);
    store8(dv + 8 * at.a, x, iv);
    store8(dv + 8 * at.b, y, iv);
  }
}

cudaError_t launch_paged_append(const PagedAppendParams& p, int dtype, cudaStream_t s) {
  const int hl = p.n_kv >= 4 ? 4 : p.n_kv >= 2 ? 2 : 1;
  const long long groups = static_cast<long long>(p.B) * p.T * hl;
  const dim3 grid(static_cast<unsigned>((groups * 8 + kThreads - 1) / kThreads));
  return dtype == GQA_CACHE_BF16 ? launch_pdl(paged_append_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, s, 0, p, hl)
                                 : launch_pdl(paged_append_kernel<uint8_t>, grid, dim3(kThreads), 0, s, 0, p, hl);
}

}  // namespace gqa
