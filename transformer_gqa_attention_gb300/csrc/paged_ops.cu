// paged_ops.cu — rotation of queries by position, the table of a rotation, and the append of new keys
// and values to their pages.
//
// All of it reads and writes every element once, and that bounds it: 8192 tokens of 32 heads (134 MB) are rotated in 22.1 us,
// 6.1 TB/s; 4 x 8192 tokens (268 MB) appended in 41.4 us, 6.5 TB/s (the copy rate).  What else costs is the chain of round
// trips of a warp that lives for one token (lengths; page, keys and values; stores) and its some 800 instructions: with
// e4m3 pages, half the bytes to write, 8 prompts of up to 2048 tokens (53 MB) take 12.5 us of which 2.2 are a launch.  There
// are warps for all B T rows: 47 % of those prompts' have no new token, read two lengths and leave.
// CTAs of 128 threads: those of 256 take 13.1, of 512 15.8.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.h"
#include "rope.cuh"

namespace gqa {

namespace {
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ uint4 ld16(const void* p) { return ld_behind_wait(static_cast<const uint4*>(p)); }
}  // namespace

// ------------------------------------------------------------------------------ rotation
// grid (ceil(n_tok / kWarps), groups of heads_each heads); a warp per token and group: eight threads
// per head, kAhead times four heads at a time, whose angles are the same.  The first heads are loaded
// while sine and cosine are computed (kAhead 1, 2, 4: 8192 tokens of 32 heads 27.1, 22.2, 22.7 us).  kAhead 1 is for
// warps of at most four heads: a few tokens, and any number of tokens that have no more (of one head 8 lanes
// of a warp's 32 have work, and each computes its eight sines and cosines itself).
template <int kAhead>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) rope_apply_kernel(const __grid_constant__ RopeParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= p.n_tok) return;  // (a whole warp)
  const int i = threadIdx.x & 7, sub = (threadIdx.x & 31) >> 3;
  const RopeLane at(p.rope, true, i);
  const int pos = __ldcg(p.positions + t);
  const int h1 = min(p.n_heads, static_cast<int>(blockIdx.y + 1) * p.heads_each);
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + t * p.stride;
  __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.out) + t * p.out_stride;
  float2 cs[8];
  const int begin = blockIdx.y * p.heads_each;
  for (int h0 = begin + sub; h0 - sub < h1; h0 += 4 * kAhead) {
    uint4 va[kAhead], vb[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (h0 + 4 * k < h1) {
        va[k] = ld16(x + (h0 + 4 * k) * 128 + 8 * at.a);
        vb[k] = ld16(x + (h0 + 4 * k) * 128 + 8 * at.b);
      }
    if (h0 - sub == begin) rope_coefficients<kAhead == 1 ? 1 : 4>(p.rope, pos, cs);  // (one: latency counts)
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (h0 + 4 * k < h1) {
        if (at.turns) {
          float a[8], b[8];
          unpack8(va[k], a);
          unpack8(vb[k], b);
          rope_turn(p.rope.layout, cs, a, b);
          va[k] = pack8(a);
          vb[k] = pack8(b);
        }
        *reinterpret_cast<uint4*>(y + (h0 + 4 * k) * 128 + 8 * at.a) = va[k];
        *reinterpret_cast<uint4*>(y + (h0 + 4 * k) * 128 + 8 * at.b) = vb[k];
      }
  }
}

// Heads of a warp: all of a token's where that gives the GPU's 152 SMs 16 warps each, else a share of them, 4 at least (the
// queries of 64 tokens, 2.2 us; all 32 heads in one warp: 4.6, eight round trips one after the other).
cudaError_t launch_rope_apply(const RopeParams& q, cudaStream_t s) {
  constexpr int kEnough = 2432;
  RopeParams p = q;
  const int parts = std::min((p.n_heads + 3) / 4, std::max(1, kEnough / p.n_tok));
  p.heads_each = ((p.n_heads + parts - 1) / parts + 3) / 4 * 4;
  const dim3 grid((p.n_tok + kWarps - 1) / kWarps, (p.n_heads + p.heads_each - 1) / p.heads_each);
  return p.heads_each <= 4 ? launch_pdl(rope_apply_kernel<1>, grid, dim3(kThreads), 0, s, 0, p)
                           : launch_pdl(rope_apply_kernel<2>, grid, dim3(kThreads), 0, s, 0, p);
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

// Eight threads per (token, head), as the rotation; kSubs heads (1, 2 or 4: what of n_kv fits) at a time, so that a
// warp holds 4 / kSubs tokens; of up to 8 heads a thread has at most two.  Everything that does not hang on
// something else is loaded first: lengths; then new keys and values, the page and the scales.
template <typename E, int kSubs>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const __grid_constant__ PagedAppendParams p) {
  constexpr bool k8 = sizeof(E) == 1;
  constexpr int kHeads = kSubs == 1 ? 1 : 2;
  griddep_launch_dependents();
  griddep_wait();
  const int group = (blockIdx.x * kThreads + threadIdx.x) >> 3;  // of eight threads
  const int i = threadIdx.x & 7;
  const int tok = group / kSubs, g0 = group - tok * kSubs;
  const int b = tok / p.T, t = tok - b * p.T;
  int n = 0, len = 0, pos = 0;
  bool live = tok < p.B * p.T;
  if (live) {
    n = p.n_new ? __ldcg(p.n_new + b) : p.T;
    len = __ldcg(p.kv_len + b);
    pos = static_cast<int>(static_cast<unsigned>(p.rope_pos ? __ldcg(p.rope_pos + b) : len) + t);  // (wraps)
    if (n < 0 || n > p.T || len < 0 || len > p.max_pages * p.pool.page_size - n) {
      if (t == 0 && g0 == 0 && i == 0) atomicOr(p.status, kDevErrRange);
      live = false;
    }
    live = live && t < n;
  }
  if (!__any_sync(0xffffffffu, live)) return;
  uint4 ka[kHeads], kb[kHeads], va[kHeads], vb[kHeads];
  float sk[kHeads], sv[kHeads];
  const RopeLane at(p.rope, p.rotate, i);
  const int s = len + t;
  const int in_table = s / p.pool.page_size;
  int page = -1;
  if (live) {
    const long long src = b * p.stride_b + t * p.stride_t;
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      const int g = g0 + h * kSubs;
      if (g < p.n_kv) {
        const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.k) + src + g * 128;
        const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v) + src + g * 128;
        ka[h] = ld16(k + 8 * at.a);
        kb[h] = ld16(k + 8 * at.b);
        va[h] = ld16(v + 8 * at.a);
        vb[h] = ld16(v + 8 * at.b);
        if (k8) {
          sk[h] = p.pool.k_scale ? __ldcg(p.pool.k_scale + g) : 1.f;
          sv[h] = p.pool.v_scale ? __ldcg(p.pool.v_scale + g) : 1.f;
        }
      }
    }
    page = __ldcg(p.page_table + static_cast<size_t>(b) * p.max_pages + in_table);
  }
  float2 cs[8];
  if (p.rotate) rope_coefficients<kSubs>(p.rope, pos, cs);
  if (!live) return;
  if (page < 0 || page >= p.pool.n_pages) {
    if (g0 == 0 && i == 0) atomicOr(p.status, kDevErrRange);
    return;
  }
  const long long row = page * p.pool.page + (s - in_table * p.pool.page_size) * p.pool.pos;
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    const int g = g0 + h * kSubs;
    if (g < p.n_kv) {
      const float ik = k8 ? 1.f / sk[h] : 1.f, iv = k8 ? 1.f / sv[h] : 1.f;
      E* dk = static_cast<E*>(p.pool.k) + row + g * p.pool.head;
      E* dv = static_cast<E*>(p.pool.v) + row + g * p.pool.head;
      float x[8], y[8];
      unpack8(ka[h], x);
      unpack8(kb[h], y);
      if (at.turns) rope_turn(p.rope.layout, cs, x, y);
      store8(dk + 8 * at.a, x, ik);
      store8(dk + 8 * at.b, y, ik);
      if constexpr (k8) {
        unpack8(va[h], x);
        unpack8(vb[h], y);
        store8(dv + 8 * at.a, x, iv);
        store8(dv + 8 * at.b, y, iv);
      } else {
        *reinterpret_cast<uint4*>(dv + 8 * at.a) = va[h];
        *reinterpret_cast<uint4*>(dv + 8 * at.b) = vb[h];
      }
    }
  }
}

template <typename E, int kSubs>
static cudaError_t launch_append(const PagedAppendParams& p, cudaStream_t s) {
  const long long threads = static_cast<long long>(p.B) * p.T * 8 * kSubs;
  return launch_pdl(paged_append_kernel<E, kSubs>, dim3(static_cast<unsigned>((threads + kThreads - 1) / kThreads)),
                    dim3(kThreads), 0, s, 0, p);
}
template <typename E>
static cudaError_t launch_append(const PagedAppendParams& p, cudaStream_t s) {
  return p.n_kv >= 4 ? launch_append<E, 4>(p, s) : p.n_kv >= 2 ? launch_append<E, 2>(p, s) : launch_append<E, 1>(p, s);
}

cudaError_t launch_paged_append(const PagedAppendParams& p, int dtype, cudaStream_t s) {
  return dtype == GQA_CACHE_BF16 ? launch_append<__nv_bfloat16>(p, s) : launch_append<uint8_t>(p, s);
}

}  // namespace gqa
