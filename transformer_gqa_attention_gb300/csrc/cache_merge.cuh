// cache_merge.cuh — what finishes the attention over caches of per-sequence length: the merge of
// units that several workers shared, and the accumulation of the key weights.
//
// Merge: pieces k of a unit give O = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k with M = max_k m_k.
// The lengths are on the device, so which units are cut is too, and the launch is made in any case.
// At most two pieces a worker, 20 MB in all: bound by latency (launch, the record, the pieces in L2),
// 3 us behind the attention of 8 ragged sequences and 26 tokens, 2 where nothing was cut.  The
// workers' blocks share a unit by rows and columns, and a block's warps its pieces where these are many,
// added up in a fixed order: results do not depend on which block is first.
//
// Weights: w[s] += sum over the four heads of 2^(c s - M) / l, from the scores that the attention left
// behind.  They can only be had once M and l are known, so the scores make a trip through memory: 64
// sequences of 8192 keys write and read 67 MB, most of it in L2 as the cache leaves it first, and update
// 17 MB of sums in 22 us behind 338 us of attention.  Blocks of 256 threads, four per SM (27 us with
// as many registers as it likes, 29 with two blocks).
#pragma once

#include <type_traits>

#include "kv_sched.h"
#include "params.h"
#include "ptx.cuh"

namespace gqa {

// Unnormalised sum of pieces k0, k0 + step, ... of a block of a cut unit's O, N float4 per lane:
// with kByRow (scratch [row][128 d], the decode step with weights) rows row0 .. row0 + rows - 1 (at
// most N), lane = float4 column; else (scratch [float4 column][row]) float4 columns col0 .. col0 +
// N - 1 of row row0 + lane.  M and l: the rows' maximum and sum; acc is relative to M.
template <bool kByRow, int N>
struct Merge {
  static constexpr int kStats = kByRow ? N : 1;
  float M[kStats], l[kStats];
  float4 acc[N];
  __device__ __forceinline__ void run(const CacheAttnParams& p, int first, int n, int row0, int rows, int col0, int k0,
                                      int step) {
    const int lane = threadIdx.x & 31;
    const int R = p.part_rows;
#pragma unroll
    for (int i = 0; i < kStats; ++i) {
      M[i] = -INFINITY;
      l[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int k = k0; k < n; k += step) {
      const size_t s = k ? partial_slot(first + k, true) : partial_slot(first, false);
      // (rows past the last read the last: loads without conditions are all in flight together)
      float2 ml[kStats];
      float4 v[N];
#pragma unroll
      for (int i = 0; i < kStats; ++i) ml[i] = __ldcg(p.part_ml + s * R + row0 + (kByRow ? min(i, rows - 1) : lane));
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const size_t at = kByRow ? (s * R + row0 + min(i, rows - 1)) * 32 + lane : (s * 32 + col0 + i) * R + row0 + lane;
        v[i] = __ldcg(reinterpret_cast<const float4*>(p.part_o) + at);
      }
      float wa[kStats], wb[kStats];
#pragma unroll
      for (int i = 0; i < kStats; ++i) {
        const float top = fmaxf(M[i], ml[i].x), tz = top == -INFINITY ? 0.f : top;
        wa[i] = fast_exp2(M[i] - tz);
        wb[i] = fast_exp2(ml[i].x - tz);
        M[i] = top;
        l[i] = l[i] * wa[i] + ml[i].y * wb[i];
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float a = wa[kByRow ? i : 0], b = wb[kByRow ? i : 0];
        acc[i] = make_float4(acc[i].x * a + v[i].x * b, acc[i].y * a + v[i].y * b, acc[i].z * a + v[i].z * b,
                             acc[i].w * a + v[i].w * b);
      }
    }
  }
};

__device__ __forceinline__ uint2 pack4(float4 v, float f) {
  return make_uint2(pack_bf16x2(v.x * f, v.y * f), pack_bf16x2(v.z * f, v.w * f));
}

// Joins the pieces of the unit that goes on past worker v's range, described by d.  A unit of n
// pieces goes on past n - 1 workers, whose blocks share it: of theirs, this is block i of `blocks`.
// A task is N rows x 128 columns with kByRow, else 32 rows x 16 columns (N = 4); ks of a block's
// eight warps share a task's pieces and add up through shared memory in a fixed order.
template <bool kByRow>
__device__ __forceinline__ void merge_unit(const CacheAttnParams& p, const int4& d, int i, int blocks) {
  constexpr int N = 4;
  __shared__ float4 sum[8][N][32];  // [warp][i][lane]
  __shared__ float2 sum_ml[8][32];  // [warp][row: i or lane]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = d.w - d.z + 1;
  const int g = d.y / p.row_groups;
  const int t0 = (d.y - g * p.row_groups) * p.group_pos;
  const int live = 4 * min(p.T - t0, p.group_pos);
  const int row_tasks = kByRow ? (live + N - 1) / N : (live + 31) / 32;
  const int tasks = kByRow ? row_tasks : 8 * row_tasks;
  // a warp for each task and share: with n - 1 workers' blocks there are enough of them
  const int ks = kByRow ? 8 : n > 8 ? 8 : n > 4 ? 4 : n > 2 ? 2 : 1;
  for (int first = i * (8 / ks); first < tasks; first += blocks * (8 / ks)) {
    const int task = first + warp / ks, share = warp % ks;
    const int row0 = (kByRow ? N : 32) * (task % row_tasks), col0 = kByRow ? 0 : N * (task / row_tasks);
    const int rows = task < tasks ? min(live - row0, kByRow ? N : 32) : 0;
    Merge<kByRow, N> m;
    m.run(p, d.z, rows > 0 && (kByRow || lane < rows) ? n : 0, row0, rows, col0, share, ks);
    if (ks > 1) {
#pragma unroll
      for (int j = 0; j < N; ++j) sum[warp][j][lane] = m.acc[j];
      if (kByRow) {
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (lane == j) sum_ml[warp][j] = make_float2(m.M[kByRow ? j : 0], m.l[kByRow ? j : 0]);
      } else {
        sum_ml[warp][lane] = make_float2(m.M[0], m.l[0]);
      }
      __syncthreads();
    }
    // element (row, float4 column) in h
    auto out = [&](int row, int col) {
      return reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.h) +
                                      (static_cast<size_t>(d.x) * p.T + t0 + (row >> 2)) * (p.n_kv * 512) +
                                      (g * 4 + (row & 3)) * 128 + 4 * col);
    };
    // the task's warp j of ks finishes element i = j, j + ks, ... of every lane
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if (ks > 1 && e % ks != share) continue;
      float4 a = m.acc[e];
      float l = m.l[kByRow ? e : 0];
      if (ks > 1) {
        const int at = kByRow ? e : lane, w0 = warp - share;
        float top = -INFINITY;
        for (int j = 0; j < ks; ++j) top = fmaxf(top, sum_ml[w0 + j][at].x);
        const float tz = top == -INFINITY ? 0.f : top;
        a = make_float4(0.f, 0.f, 0.f, 0.f);
        l = 0.f;
        for (int j = 0; j < ks; ++j) {
          const float2 ml = sum_ml[w0 + j][at];
          const float f = fast_exp2(ml.x - tz);
          const float4 v = sum[w0 + j][e][lane];
          a = make_float4(a.x + f * v.x, a.y + f * v.y, a.z + f * v.z, a.w + f * v.w);
          l += f * ml.y;
        }
      }
      if (kByRow ? e < rows : lane < rows)
        *(kByRow ? out(row0 + e, lane) : out(row0 + lane, col0 + e)) = pack4(a, l == 0.f ? 0.f : 1.f / l);
    }
    if (ks > 1) __syncthreads();
  }
}

__global__ void __launch_bounds__(256) cache_merge_kernel(const CacheAttnParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int v = blockIdx.x;
  const int4 d = __ldcg(p.merge + v);
  const int st = *reinterpret_cast<volatile const int*>(p.status);
  // after a wait that ran out the scratch may be unwritten
  if (d.x < 0 || (st & kDevErrTimeout)) return;
  merge_unit<false>(p, d, (v - d.z) * gridDim.y + blockIdx.y, (d.w - d.z) * gridDim.y);
}

// (maximum, sum) of four heads from 16-byte aligned memory.
__device__ __forceinline__ void load_ml(const float2* at, float2 (&m)[4]) {
  const float4 a = __ldcg(reinterpret_cast<const float4*>(at)), b = __ldcg(reinterpret_cast<const float4*>(at) + 1);
  m[0] = make_float2(a.x, a.y);
  m[1] = make_float2(a.z, a.w);
  m[2] = make_float2(b.x, b.y);
  m[3] = make_float2(b.z, b.w);
}

__device__ __forceinline__ float2 join_ml(float2 a, float2 b) {
  const float top = fmaxf(a.x, b.x), tz = top == -INFINITY ? 0.f : top;
  return make_float2(top, a.y * fast_exp2(a.x - tz) + b.y * fast_exp2(b.x - tz));
}

// The decode step with key weights: blocks 0 .. workers - 1 merge, the others add each key's
// weight, the sum over the four heads of 2^(c s - M) / l, to the running sums, one key tile per warp
// at a time.
__global__ void __launch_bounds__(256, 4) cache_weights_kernel(const CacheAttnParams p, int workers) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_launch_dependents();
  griddep_wait();
  if (blockIdx.x < workers) {
    const int v = blockIdx.x;
    const int4 d = __ldcg(p.merge + v);
    const int st = *reinterpret_cast<volatile const int*>(p.status);
    if (d.x >= 0 && !(st & kDevErrTimeout)) merge_unit<true>(p, d, v - d.z, d.w - d.z);
    return;
  }
  const int total = __ldcg(p.total_tiles);
  const int n_warps = (gridDim.x - workers) * 8;
  const int R = p.part_rows;
  if (*reinterpret_cast<volatile const int*>(p.status) & kDevErrTimeout) return;
  // neighbouring warps have neighbouring tiles
  for (int i = (blockIdx.x - workers) * 8 + warp; i < total; i += n_warps) {
    const int4 tu = __ldcg(p.tile_unit + i);
    float4 x[4];  // keys 32 k + lane, their four heads' scores
#pragma unroll
    for (int k = 0; k < 4; ++k)
      x[k] = __ldcg(reinterpret_cast<const float4*>(p.scores) + static_cast<size_t>(i) * kKvTile + 32 * k + lane);
    float* w = p.weights + static_cast<size_t>(tu.x) * p.S_max + tu.y * kKvTile;
    bool seen[4];
    float a[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // -inf in all four heads: past the end (or of no weight)
      seen[k] = x[k].x != -INFINITY || x[k].y != -INFINITY || x[k].z != -INFINITY || x[k].w != -INFINITY;
      a[k] = seen[k] ? __ldcg(w + 32 * k + lane) : 0.f;
    }
    // the heads' maxima and sums: the unit's, or of its pieces joined
    float2 m[4];
    if (tu.z == tu.w) {
      load_ml(p.unit_ml + tu.x * 4, m);
    } else {
#pragma unroll
      for (int h = 0; h < 4; ++h) m[h] = make_float2(-INFINITY, 0.f);
      const int n = tu.w - tu.z + 1;
      const bool shared = n > 8;  // many pieces: the lanes share them
      for (int k = shared ? lane : 0; k < n; k += shared ? 32 : 1) {
        float2 o[4];
        load_ml(p.part_ml + static_cast<size_t>(k ? partial_slot(tu.z + k, true) : partial_slot(tu.z, false)) * R, o);
#pragma unroll
        for (int h = 0; h < 4; ++h) m[h] = join_ml(m[h], o[h]);
      }
      if (shared) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
          for (int h = 0; h < 4; ++h)
            m[h] = join_ml(m[h], make_float2(__shfl_xor_sync(0xffffffffu, m[h].x, o), __shfl_xor_sync(0xffffffffu, m[h].y, o)));
      }
    }
    float inv[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      inv[h] = 1.f / m[h].y;
      if (m[h].x == -INFINITY) m[h].x = 0.f;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float add = fast_exp2(fmaf(x[k].x, p.scale_log2, -m[0].x)) * inv[0] +
                        fast_exp2(fmaf(x[k].y, p.scale_log2, -m[1].x)) * inv[1] +
                        fast_exp2(fmaf(x[k].z, p.scale_log2, -m[2].x)) * inv[2] +
                        fast_exp2(fmaf(x[k].w, p.scale_log2, -m[3].x)) * inv[3];
      if (seen[k]) w[32 * k + lane] = a[k] + add;
    }
  }
}

}  // namespace gqa
