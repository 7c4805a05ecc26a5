// paged_attn.cuh — attention of one new token per sequence over a paged cache.
//
// A CTA per (sequence, kv head); a warp takes every eighth key, a lane four elements of it.  The
// four query heads of the kv head share each key and value; online softmax in fp32, the warps'
// results joined through shared memory.
#pragma once

#include <cuda_fp8.h>

#include "params.h"
#include "ptx.cuh"

namespace gqa {

__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 v = __ldcg(reinterpret_cast<const uint2*>(p));
  return make_float4(bf16lo_to_f32(v.x), bf16hi_to_f32(v.x), bf16lo_to_f32(v.y), bf16hi_to_f32(v.y));
}
__device__ __forceinline__ float4 load4(const uint8_t* p) {
  const uint32_t v = __ldcg(reinterpret_cast<const uint32_t*>(p));
  const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v & 0xFFFF), __NV_E4M3);
  const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v >> 16), __NV_E4M3);
  const float2 x = __half22float2(__half2(a)), y = __half22float2(__half2(b));
  return make_float4(x.x, x.y, y.x, y.y);
}

template <typename E>
__global__ void __launch_bounds__(256) paged_attn_kernel(const __grid_constant__ PagedAttnParams p) {
  __shared__ float4 red_o[8][4][32];
  __shared__ float2 red_ml[8][4];
  griddep_launch_dependents();
  griddep_wait();
  const int g = blockIdx.x, b = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = __ldcg(p.kv_len + b);
  const bool in_range = len >= 0 && len <= p.max_pages * p.pool.page_size - p.n_new;
  const int end = in_range ? len + p.n_new : 0;
  const float ks = p.scale_log2 * (p.pool.k_scale ? __ldg(p.pool.k_scale + g) : 1.f);
  float4 q[4], o[4];
  float m[4], l[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    q[h] = load4(static_cast<const __nv_bfloat16*>(p.q) + (static_cast<size_t>(b) * p.n_kv * 4 + g * 4 + h) * 128 + 4 * lane);
    o[h] = make_float4(0.f, 0.f, 0.f, 0.f);
    m[h] = -INFINITY;
    l[h] = 0.f;
  }
  bool bad = !in_range;
  for (int s = warp; s < end; s += 8) {
    const int n = s / p.pool.page_size;
    const int page = __ldcg(p.page_table + static_cast<size_t>(b) * p.max_pages + n);
    if (page < 0 || page >= p.pool.n_pages) {
      bad = true;
      break;
    }
    const long long at = page * p.pool.page + (s - n * p.pool.page_size) * p.pool.pos + g * p.pool.head + 4 * lane;
    const float4 k = load4(static_cast<const E*>(p.pool.k) + at), v = load4(static_cast<const E*>(p.pool.v) + at);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      float x = q[h].x * k.x + q[h].y * k.y + q[h].z * k.z + q[h].w * k.w;
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
      x *= ks;
      const float top = fmaxf(m[h], x), base = top == -INFINITY ? 0.f : top;
      const float a = fast_exp2(m[h] - base), e = fast_exp2(x - base);
      m[h] = top;
      l[h] = l[h] * a + e;
      o[h] = make_float4(o[h].x * a + e * v.x, o[h].y * a + e * v.y, o[h].z * a + e * v.z, o[h].w * a + e * v.w);
    }
  }
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    red_o[warp][h][lane] = o[h];
    if (lane == 0) red_ml[warp][h] = make_float2(m[h], l[h]);
  }
  bad = __syncthreads_or(bad);
  if (bad && threadIdx.x == 0) atomicOr(p.status, kDevErrRange);
  if (warp >= 4) return;
  float M = -INFINITY, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int w = 0; w < 8; ++w) M = fmaxf(M, red_ml[w][warp].x);
  const float base = M == -INFINITY ? 0.f : M;
  for (int w = 0; w < 8; ++w) {
    const float f = fast_exp2(red_ml[w][warp].x - base);
    const float4 v = red_o[w][warp][lane];
    L += f * red_ml[w][warp].y;
    acc = make_float4(acc.x + f * v.x, acc.y + f * v.y, acc.z + f * v.z, acc.w + f * v.w);
  }
  float inv = end == 0 ? 0.f : (p.pool.v_scale ? __ldg(p.pool.v_scale + g) : 1.f) / L;
  if (bad) inv = __int_as_float(0x7fc00000);
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.h) + (static_cast<size_t>(b) * p.n_kv * 4 + g * 4 + warp) * 128 +
                            4 * lane) = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

}  // namespace gqa
