// cache_ops.cu — upkeep of the key / value cache [B, S_max, n_kv, 128]: the accepted path of a
// drafted tree moved to the front of its drafted positions, and eviction by accumulated weight
// (selection of the positions to keep, then their move).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "launch.h"
#include "ptx.cuh"

namespace gqa {

// ------------------------------------------------------------------------------ commit
constexpr int kCommitThreads = 256;
constexpr int kCommitSlices = 8;  // CTAs (one cluster) per sequence; each moves 1/8 of every row

// Rows prefix + path[i] -> prefix + i of both caches.  path is strictly increasing, so path[i] >=
// i: every row moves towards the front, and the rows of one step are read before any is written.
__global__ void __launch_bounds__(kCommitThreads) cache_commit_kernel(const CommitParams p) {
  griddep_wait();
  const int b = blockIdx.y, slice = blockIdx.x;
  const int prefix = __ldcg(p.prefix_len + b);
  const int n = __ldcg(p.n_accept + b);
  const int* path = p.path + static_cast<size_t>(b) * p.T;
  bool ok = prefix >= 0 && prefix <= p.S_max - p.T && n >= 0 && n <= p.T;
  if (ok) {
    for (int i = threadIdx.x; i < n; i += kCommitThreads) {
      const int at = __ldcg(path + i);
      ok = ok && at >= i && at < p.T && (i == 0 || __ldcg(path + i - 1) < at);
    }
  }
  ok = __syncthreads_and(ok);
  if (ok) {
    // 16-byte chunks of a row: n_kv x 16 of K, then as many of V; this CTA's are slice, slice + 8, ...
    const int per_cache = p.n_kv * 16;
    const int mine = 2 * per_cache / kCommitSlices;
    const size_t row_chunks = per_cache;
    const size_t base = (static_cast<size_t>(b) * p.S_max + prefix) * row_chunks;
    const int rows_per_step = kCommitThreads / mine;  // n_kv <= 8: at least 8
    const int r = threadIdx.x / mine;
    const int c = (threadIdx.x % mine) * kCommitSlices + slice;
    uint4* cache = static_cast<uint4*>(c < per_cache ? p.k : p.v) + base + (c < per_cache ? c : c - per_cache);
    for (int i0 = 0; i0 < n; i0 += rows_per_step) {
      const int i = i0 + r;
      const bool live = r < rows_per_step && i < n;
      uint4 v{};
      if (live) v = cache[static_cast<size_t>(__ldcg(path + i)) * row_chunks];
      __syncthreads();
      if (live) cache[static_cast<size_t>(i) * row_chunks] = v;
      __syncthreads();
    }
  }
  cluster_sync();  // every CTA of the sequence has read its length
  if (slice == 0 && threadIdx.x == 0) {
    if (!ok) atomicOr(p.status, kDevErrRange);
    p.new_len[b] = ok ? prefix + n : prefix;
  }
}

cudaError_t launch_cache_commit(const CommitParams& p, cudaStream_t s) {
  return launch_pdl(cache_commit_kernel, dim3(kCommitSlices, p.B), dim3(kCommitThreads), 0, s, kCommitSlices, p);
}

// ------------------------------------------------------------------------------ eviction
constexpr int kSelThreads = 1024;

// Order-preserving unsigned image of a weight: larger weight, larger image; -0 equals +0, and a
// NaN comes below everything.
__device__ __forceinline__ uint32_t weight_rank(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum of `v` over the CTA's threads; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = lane < kSelThreads / 32 ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  *total = warp_sums[kSelThreads / 32 - 1];
  const int before = (warp ? warp_sums[warp - 1] : 0) + x - v;
  __syncthreads();
  return before;
}

// One CTA per (kv group, sequence): the positions to keep, ascending, and their weights.  The
// weight of the last one picked is found digit by digit (four 8-bit counts), then one ordered
// pass emits everything above it and the first of its equals.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
  __shared__ int hist[256];
  __shared__ int warp_sums[32];
  __shared__ int sh_digit, sh_need;
  griddep_wait();
  const int g = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const size_t unit = static_cast<size_t>(b) * p.n_kv + g;
  const float* w = p.weights + unit * p.S_max;
  float* ow = p.out_weights + unit * p.S_out;
  int* kept = p.kept + unit * p.budget;
  const int len = __ldcg(p.kv_len + b);
  if (len < 0 || len > p.S_max) {
    if (tid == 0) atomicOr(p.status, kDevErrRange);
    for (int i = tid; i < p.budget; i += kSelThreads) kept[i] = -1;
    return;
  }
  const int n_keep = min(len, p.budget);
  const int lo = p.n_first, hi = len - p.n_recent;  // the middle, of which the heaviest stay
  uint32_t thr = 0;
  int eq_take = 0;
  if (len > p.budget) {
    int need = p.budget - p.n_first - p.n_recent;
    if (need > 0) {
      uint32_t prefix = 0, pmask = 0;
      for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        for (int s = lo + tid; s < hi; s += kSelThreads) {
          const uint32_t u = weight_rank(__ldcg(w + s));
          if ((u & pmask) == prefix) atomicAdd(&hist[(u >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
          int d = 255, n = need;
          while (hist[d] < n) n -= hist[d--];
          sh_digit = d;
          sh_need = n;
        }
        __syncthreads();
        prefix |= static_cast<uint32_t>(sh_digit) << shift;
        pmask |= 255u << shift;
        need = sh_need;
        __syncthreads();
      }
      thr = prefix;
      eq_take = need;
    } else {
      thr = 0xFFFFFFFFu;  // nothing of the middle stays (no rank is this high)
    }
  }
  int out = 0, eq_seen = 0;
  for (int s0 = 0; s0 < len; s0 += kSelThreads) {
    const int s = s0 + tid;
    float x = 0.f;
    bool gt = false, eq = false;
    if (s < len) {
      x = __ldcg(w + s);
      if (len <= p.budget || s < lo || s >= hi) {
        gt = true;
      } else {
        const uint32_t u = weight_rank(x);
        gt = u > thr;
        eq = u == thr;
      }
    }
    int n_eq;
    const int eq_at = eq_seen + block_scan(eq, warp_sums, &n_eq);
    const bool take = gt || (eq && eq_at < eq_take);
    int n_take;
    const int at = out + block_scan(take, warp_sums, &n_take);
    if (take) {  // at <= s: in place, only positions already read are written
      kept[at] = s;
      ow[at] = x;
    }
    out += n_take;
    eq_seen += n_eq;
  }
  __syncthreads();
  for (int i = n_keep + tid; i < p.budget; i += kSelThreads) kept[i] = -1;
  // weights of what is decoded next start from zero
  const int zero_to = p.in_place ? len : p.S_out;
  for (int i = n_keep + tid; i < zero_to; i += kSelThreads) ow[i] = 0.f;
}

constexpr int kMoveThreads = 256;
constexpr int kMoveChunk = 4;   // 16-byte pieces of a row that one CTA moves
constexpr int kMoveRows = 4;    // rows in flight per thread

// One CTA per (64-byte column slice of K or V, kv group, sequence): rows kept[i] -> i.  kept is
// ascending, so kept[i] >= i; in place, a step's rows are all read before any is written, and no
// later step reads a row that it wrote.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p) {
  griddep_wait();
  const int slice = blockIdx.x, g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int per_cache = 16 / kMoveChunk;
  const bool is_v = slice >= per_cache;
  const size_t unit = static_cast<size_t>(b) * p.n_kv + g;
  const int* kept = p.kept + unit * p.budget;
  const int c = (slice - (is_v ? per_cache : 0)) * kMoveChunk + tid % kMoveChunk;
  const size_t row = static_cast<size_t>(p.n_kv) * 16;
  const uint4* src = static_cast<const uint4*>(is_v ? p.v : p.k) + (static_cast<size_t>(b) * p.S_max * p.n_kv + g) * 16 + c;
  uint4* dst = static_cast<uint4*>(is_v ? p.out_v : p.out_k) + (static_cast<size_t>(b) * p.S_out * p.n_kv + g) * 16 + c;
  constexpr int kStep = kMoveThreads / kMoveChunk;
  for (int i0 = 0; i0 < p.budget; i0 += kStep * kMoveRows) {
    uint4 v[kMoveRows];
    int from[kMoveRows];
#pragma unroll
    for (int j = 0; j < kMoveRows; ++j) {
      const int i = i0 + j * kStep + tid / kMoveChunk;
      from[j] = i < p.budget ? __ldcg(kept + i) : -1;
    }
#pragma unroll
    for (int j = 0; j < kMoveRows; ++j)
      if (from[j] >= 0) v[j] = __ldcg(src + from[j] * row);
    if (p.in_place) __syncthreads();
#pragma unroll
    for (int j = 0; j < kMoveRows; ++j) {
      const int i = i0 + j * kStep + tid / kMoveChunk;
      if (from[j] >= 0) dst[i * row] = v[j];
    }
  }
  if (slice == 0 && g == 0) {
    for (int i = tid; i <= p.budget; i += kMoveThreads) {
      const bool here = i < p.budget && __ldcg(kept + i) >= 0;
      if (!here && (i == 0 || __ldcg(kept + i - 1) >= 0)) p.new_len[b] = i;
    }
  }
}

cudaError_t launch_evict_select(const EvictParams& p, cudaStream_t s) {
  return launch_pdl(evict_select_kernel, dim3(p.n_kv, p.B), dim3(kSelThreads), 0, s, 0, p);
}

cudaError_t launch_evict_move(const EvictParams& p, cudaStream_t s) {
  return launch_pdl(evict_move_kernel, dim3(2 * 16 / kMoveChunk, p.n_kv, p.B), dim3(kMoveThreads), 0, s, 0, p);
}

}  // namespace gqa
