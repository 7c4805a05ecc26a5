// cache_ops.cu — upkeep of the key / value cache [B, S_max, n_kv, 128]: the accepted path of a
// drafted tree moved to the front of its drafted positions, and eviction by accumulated weight
// (selection of the positions to keep, then their move).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.h"
#include "ptx.cuh"

namespace gqa {

// ------------------------------------------------------------------------------ commit
constexpr int kCommitThreads = 256;
constexpr int kCommitSlices = 8;  // CTAs (one cluster) per sequence; each moves 1/8 of every row

// Rows prefix + path[i] -> prefix + i of both caches.  path is strictly increasing, so path[i] >=
// i: every row moves towards the front, and the rows of one step are read before any is written.
// An accepted path has a few tokens, one step of the loop: a launch is what that costs (2.6 us in a graph for
// 1 and for 64 sequences), so the slices of a row are CTAs of their own, and the length, which may be
// written over, is written once the cluster has read it.  Long paths are bound by the steps' round trips, 8
// rows each with 8 kv heads: 128 tokens of one sequence take 18 us, 256 (2 MB) 34, 128 of 64 sequences (67 MB)
// 32, of 256 sequences (268 MB) 105.
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
constexpr int kSelThreads = 512;
constexpr int kSelEach = 12;                         // positions per thread of a staged chunk (a multiple of 4)
constexpr int kSelChunk = kSelThreads * kSelEach;
constexpr int kSelBins = 2048;
constexpr int kSelMaxCluster = 8;

// Order-preserving unsigned image of a weight: larger weight, larger image; -0 equals +0, and a
// NaN comes below everything.
__device__ __forceinline__ uint32_t weight_rank(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum of `v` over the CTA's threads; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  constexpr int kWarps = kSelThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int before = x - v, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int s = warp_sums[w];
    if (w < warp) before += s;
    all += s;
  }
  *total = all;
  __syncthreads();
  return before;
}

// The positions that a (sequence, kv head) keeps, ascending.  A cluster of gridDim.x CTAs shares its
// positions, each a contiguous slice.  The rank that the last kept weight has is found in digits of
// 11, 11 and 10 bits: every CTA counts its slice's digits in shared memory, sums the cluster's
// counts through distributed shared memory and finds the digit; once all of a digit's positions are
// wanted the search ends early.  Then everything above is kept, and the first of the equal ones: a
// position's place is the number kept before it, a prefix sum over the slice and the CTAs before.
// Reads each weight once (a slice stays in shared memory; only heads of more than 49152 positions read it
// five times) and is bound by the passes' barriers and shared-memory atomics: 7 us of the 8.9 that
// one sequence of 4100 positions takes, 18 of 140 for 32 of up to 8192.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
  __shared__ __align__(16) float stage[kSelChunk];
  __shared__ __align__(16) int hist[kSelBins];
  __shared__ int warp_sums[kSelThreads / 32];
  __shared__ int found[3];   // digit, still wanted of it, its count
  __shared__ int totals[2];  // of the slice: kept for sure, equal
  griddep_wait();
  const int rank = blockIdx.x, n_ctas = gridDim.x, g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const size_t unit = static_cast<size_t>(b) * p.n_kv + g;
  const float* w = p.weights + unit * p.S_max;
  int* kept = p.kept + unit * p.budget;
  const int len = __ldcg(p.kv_len + b);
  const bool bad = len < 0 || len > p.S_max;
  if (rank == 0 && tid == 0) {
    if (g == 0) p.old_len[b] = bad ? -1 : len;
    if (bad) atomicOr(p.status, kDevErrRange);
  }
  if (bad || len <= p.budget) {  // the same for the whole cluster
    for (int i = rank * kSelThreads + tid; i < p.budget; i += n_ctas * kSelThreads) kept[i] = !bad && i < len ? i : -1;
    return;
  }
  const int per = (len + n_ctas - 1) / n_ctas;
  const int lo = min(len, rank * per), hi = min(len, lo + per);
  const int mid0 = p.n_first, mid1 = len - p.n_recent;  // the heaviest of these stay
  const bool staged = per <= kSelChunk;
  auto load_chunk = [&](int s0) {
    float v[kSelEach];  // (without conditions, so that all are in flight together)
#pragma unroll
    for (int q = 0; q < kSelEach; ++q) v[q] = __ldcg(w + min(s0 + q * kSelThreads + tid, hi - 1));
#pragma unroll
    for (int q = 0; q < kSelEach; ++q) stage[q * kSelThreads + tid] = v[q];
    __syncthreads();
  };
  auto sync_all = [&] {
    if (n_ctas > 1)
      cluster_sync();
    else
      __syncthreads();
  };
  if (staged) load_chunk(lo);

  // ranks above prefix | ~mask stay, and the first `rem` of those whose masked bits are prefix
  uint32_t prefix = 0xFFFFFFFFu, mask = 0xFFFFFFFFu;  // (no weight has this rank: none)
  int rem = p.budget - p.n_first - p.n_recent;
  if (rem > 0) {
    prefix = mask = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t digit_mask = pass == 2 ? 1023u : 2047u;
      for (int i = tid; i < kSelBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int s = max(lo, mid0) + tid; s < min(hi, mid1); s += kSelThreads) {
        const uint32_t u = weight_rank(staged ? stage[s - lo] : __ldcg(w + s));
        if ((u & mask) == prefix) atomicAdd(&hist[(u >> shift) & digit_mask], 1);
      }
      sync_all();
      // thread t: bins from the top, 4 t .. 4 t + 3
      const int top = kSelBins - 4 - 4 * tid;
      int4 c = make_int4(0, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < kSelMaxCluster; ++r) {
        if (r < n_ctas) {
          const int4 o = r == rank ? *reinterpret_cast<const int4*>(hist + top)
                                   : ld_shared_cluster_int4(mapa_shared(smem_u32(hist + top), r));
          c = make_int4(c.x + o.x, c.y + o.y, c.z + o.z, c.w + o.w);
        }
      }
      int all;
      int above = block_scan(c.x + c.y + c.z + c.w, warp_sums, &all);
      const int n[4] = {c.w, c.z, c.y, c.x};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (above < rem && rem <= above + n[k]) {
          found[0] = top + 3 - k;
          found[1] = rem - above;
          found[2] = n[k];
        }
        above += n[k];
      }
      sync_all();  // found is written, and the counts of this CTA have been read
      prefix |= static_cast<uint32_t>(found[0]) << shift;
      mask |= digit_mask << shift;
      rem = found[1];
      if (found[2] == rem) break;
    }
  }
  const uint32_t above = prefix | ~mask;
  // flags of the thread's positions of a staged chunk: bits 0..15 kept for sure, 16..31 equal
  auto flags = [&](int s0) {
    uint32_t f = 0;
#pragma unroll
    for (int q = 0; q < kSelEach; q += 4) {
      const float4 v = *reinterpret_cast<const float4*>(stage + tid * kSelEach + q);
      const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int s = s0 + tid * kSelEach + q + k;
        if (s < hi) {
          const uint32_t u = weight_rank(x[k]);
          const bool edge = s < mid0 || s >= mid1;
          if (edge || u > above)
            f |= 1u << (q + k);
          else if ((u & mask) == prefix)
            f |= 0x10000u << (q + k);
        }
      }
    }
    return f;
  };
  auto packed = [](uint32_t f) { return (__popc(f & 0xFFFFu) << 16) | __popc(f >> 16); };  // at most kSelChunk each
  // this slice's totals, then those of the CTAs before it
  int sure = 0, equal = 0;
  uint32_t f = 0;
  int before = 0;
  for (int s0 = lo; s0 < hi; s0 += kSelChunk) {
    if (!staged) {
      __syncthreads();
      load_chunk(s0);
    }
    f = flags(s0);
    int all;
    before = block_scan(packed(f), warp_sums, &all);
    sure += all >> 16;
    equal += all & 0xFFFF;
  }
  int base_sure = 0, base_equal = 0;
  if (n_ctas > 1) {
    if (tid == 0) {
      totals[0] = sure;
      totals[1] = equal;
    }
    cluster_sync();
    for (int r = 0; r < rank; ++r) {
      base_sure += ld_shared_cluster_int(mapa_shared(smem_u32(&totals[0]), r));
      base_equal += ld_shared_cluster_int(mapa_shared(smem_u32(&totals[1]), r));
    }
  }
  for (int s0 = lo; s0 < hi; s0 += kSelChunk) {
    if (!staged) {
      __syncthreads();
      load_chunk(s0);
      f = flags(s0);
      int all;
      before = block_scan(packed(f), warp_sums, &all);
      sure = all >> 16;  // of this chunk
      equal = all & 0xFFFF;
    }
    int gt = base_sure + (before >> 16), eq = base_equal + (before & 0xFFFF);
#pragma unroll
    for (int k = 0; k < kSelEach; ++k) {
      const bool is_gt = (f >> k) & 1u, is_eq = (f >> (16 + k)) & 1u;
      if (is_gt || (is_eq && eq < rem)) kept[gt + min(eq, rem)] = s0 + tid * kSelEach + k;
      gt += is_gt;
      eq += is_eq;
    }
    base_sure += sure;
    base_equal += equal;
  }
  if (n_ctas > 1) cluster_sync();  // no CTA leaves while another reads its totals
}

constexpr int kMoveThreads = 256;
constexpr int kMovePieces = 4;   // 16-byte pieces of a row that one CTA moves
constexpr int kMoveRows = 8;     // rows in flight per thread
constexpr int kMoveStep = kMoveThreads / kMovePieces;
constexpr int kMoveChunk = kMoveStep * kMoveRows;  // rows of a CTA's step
constexpr int kMoveSlices = 2 * 16 / kMovePieces;  // of K and V; one more block moves the weights

// Rows kept[i] -> i: one CTA per (64-byte column slice of K or V, kv group, sequence), or several
// that take steps in turn when the outputs are other buffers.  kept is ascending, so kept[i] >= i; in
// place, a step's rows are all read before any is written, and no later step reads a row that it
// wrote.  For a batch bound by memory: up to 4096 of up to 8192 positions of 32 sequences (820 MB) to other
// buffers in 122 us, 6.7 TB/s.  For one sequence in place by the steps, which one CTA takes one after another
// (whole evictions, us, other buffers / in place, 8 kv heads: 4100 to 1024 positions 11 / 12, 32768 to 16384
// 47 / 70; one kv head: 32768 to 16384 25 / 61; without the one CTA that moves a head's weights 44 and 22 to other
// buffers, the others the same).
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p) {
  griddep_wait();
  const int slice = blockIdx.x % (kMoveSlices + 1), part = blockIdx.x / (kMoveSlices + 1), g = blockIdx.y, b = blockIdx.z;
  const int parts = gridDim.x / (kMoveSlices + 1), tid = threadIdx.x;
  const size_t unit = static_cast<size_t>(b) * p.n_kv + g;
  const int* kept = p.kept + unit * p.budget;
  if (slice == kMoveSlices) {  // weights, and the new length
    if (part > 0) return;
    const float* w = p.weights + unit * p.S_max;
    float* ow = p.out_weights + unit * p.S_out;
    for (int i0 = 0; i0 < p.budget; i0 += kMoveThreads * kMoveRows) {
      float v[kMoveRows];
      int from[kMoveRows];
#pragma unroll
      for (int j = 0; j < kMoveRows; ++j) {
        const int i = i0 + j * kMoveThreads + tid;
        from[j] = i < p.budget ? __ldcg(kept + i) : -1;
      }
#pragma unroll
      for (int j = 0; j < kMoveRows; ++j) v[j] = __ldcg(w + max(from[j], 0));
      if (p.in_place) __syncthreads();
#pragma unroll
      for (int j = 0; j < kMoveRows; ++j)
        if (from[j] >= 0) ow[i0 + j * kMoveThreads + tid] = v[j];
    }
    // weights of what is decoded next start from zero
    const int old_len = __ldcg(p.old_len + b);
    const int n_keep = min(old_len, p.budget);
    if (old_len >= 0) {
      const int zero_to = p.in_place ? old_len : p.S_out;
      for (int i = n_keep + tid; i < zero_to; i += kMoveThreads) ow[i] = 0.f;
    }
    if (g == 0 && tid == 0) p.new_len[b] = max(n_keep, 0);
    return;
  }
  const int per_cache = kMoveSlices / 2;
  const bool is_v = slice >= per_cache;
  const int c = (slice - (is_v ? per_cache : 0)) * kMovePieces + tid % kMovePieces;
  const size_t row = static_cast<size_t>(p.n_kv) * 16;
  const uint4* src = static_cast<const uint4*>(is_v ? p.v : p.k) + (static_cast<size_t>(b) * p.S_max * p.n_kv + g) * 16 + c;
  uint4* dst = static_cast<uint4*>(is_v ? p.out_v : p.out_k) + (static_cast<size_t>(b) * p.S_out * p.n_kv + g) * 16 + c;
  for (int i0 = part * kMoveChunk; i0 < p.budget; i0 += parts * kMoveChunk) {
    uint4 v[kMoveRows];
    int from[kMoveRows];
#pragma unroll
    for (int j = 0; j < kMoveRows; ++j) {
      const int i = i0 + j * kMoveStep + tid / kMovePieces;
      from[j] = i < p.budget ? __ldcg(kept + i) : -1;
      if (p.in_place && from[j] == i) from[j] = -1;  // already there
    }
#pragma unroll
    for (int j = 0; j < kMoveRows; ++j)
      if (from[j] >= 0) v[j] = __ldcg(src + from[j] * row);
    if (p.in_place) __syncthreads();
#pragma unroll
    for (int j = 0; j < kMoveRows; ++j) {
      const int i = i0 + j * kMoveStep + tid / kMovePieces;
      if (from[j] >= 0) dst[i * row] = v[j];
    }
  }
}

cudaError_t launch_evict_select(const EvictParams& p, cudaStream_t s) {
  // As few CTAs per (sequence, kv head) as hold its positions in their shared memory (up to eight),
  // since every exchange between them costs more than it saves below that.  Measured with 1, 2, 4, 8
  // CTAs (whole eviction, us): one sequence of 4100 positions 8.8, 10.8, 12.0, 15.3; of 16384 33.4, 25.9,
  // 16.2, 18.7; of 32768 83, 53, 40, 28; 16 sequences of 4096 49, 53, 67, 118.
  int c = 1;
  while (c < kSelMaxCluster && (p.S_max + c - 1) / c > kSelChunk) c *= 2;
  return launch_pdl(evict_select_kernel, dim3(c, p.n_kv, p.B), dim3(kSelThreads), 0, s, c > 1 ? c : 0, p);
}

cudaError_t launch_evict_move(const EvictParams& p, cudaStream_t s) {
  // in place the steps of a slice follow one another in one CTA; else about 1024 CTAs share them
  const long long units = static_cast<long long>(p.B) * p.n_kv;
  const int steps = (p.budget + kMoveChunk - 1) / kMoveChunk;
  const int parts = p.in_place ? 1 : static_cast<int>(std::max(1LL, std::min<long long>(steps, 1024 / (units * kMoveSlices))));
  return launch_pdl(evict_move_kernel, dim3(parts * (kMoveSlices + 1), p.n_kv, p.B), dim3(kMoveThreads), 0, s, 0, p);
}

}  // namespace gqa
