// cache_attn_few.cuh — attention of at most 16 positions per sequence over caches whose lengths
// differ from sequence to sequence (cache_roles.cuh has the CTA's roles): small drafted trees, and
// the decode step that hands on its scores.
//
// With 4 T <= 64 rows (position, head) the products are turned round, so that the 128 keys of a
// tile fill the tensor core's rows and no lane idles for want of queries:
//   S^T = K Q^T    [128 keys, rows]: one softmax thread per key, its scores of all rows in registers
//   O^T = V^T P    [128 d, rows]: V as stored (d contiguous), P [keys][rows] from shared memory
// A thread then does 4 T exponentials per tile where a thread per row would do 128.  The row
// maxima, which lie across threads here, are only needed to keep 2^(c s - m) in range: a tile whose
// scores all stay below m + 8 (one vote per tile) leaves m as it is; otherwise m is reduced across
// the slot's threads and O and l are rescaled.  l is kept per thread and summed once a piece.
// Each softmax slot is a worker with its own range of tiles.
//
// TMEM columns (64 each): S_0, S_1, O_0, O_1.
#pragma once

#include "cache_roles.cuh"

namespace gqa {

struct CacheFewSmem {
  static constexpr int kQHalf = 64 * 128;       // 64 rows x 64 columns
  static constexpr int kPBytes = 128 * 128;     // P: 128 keys x 64 rows, 128-byte swizzle
  static constexpr int kP = 4 * kQHalf;         // behind the slots' queries
  static constexpr int kK = kP + 2 * kPBytes;
  static constexpr int kV = kK + kKStages * kKvTileBytes;
  static constexpr int kBar = kV + kVStages * kKvTileBytes;
  static constexpr int kRanges = kBar + CacheBars::kBytes;
  static constexpr int kStats = kRanges + CacheRanges::kBytes;  // per slot [64] each: m or 0, m + 8, factors
  static constexpr int kBytes = kStats + 2 * 3 * 64 * 4 + 1024;
};

struct OpMax {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct OpSum {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};

// Reduces N (<= 32, a power of two) columns over the warp's lanes: each step a lane passes on half
// of its columns and keeps the other half.  The result of one column ends in v[0]; returns which.
template <int N, typename Op>
__device__ __forceinline__ int reduce_columns(float (&v)[N], Op op) {
  const int lane = threadIdx.x & 31;
  int col = 0;
  int n = N;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        if (i < n) {
          const float send = up ? v[i] : v[i + n];
          const float keep = up ? v[i + n] : v[i];
          v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
      }
      if (up) col += n;
    } else {
      v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    }
  }
  return col;
}

// kCols: rows of the product the softmax works on (4: one position; 16, 32, 64: up to 4, 8, 16).
template <int kCols, bool kScores>
__global__ void __launch_bounds__(384, 1)
    cache_attn_few_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const CacheAttnParams p) {
  static_assert(!kScores || kCols == 4, "scores are handed on for one position per sequence");
  using L = CacheFewSmem;
  constexpr int kWork = 2;
  constexpr int kN = kCols < 16 ? 16 : kCols;       // N of S^T (a multiple of 16)
  constexpr int kChunk = kCols < 32 ? kCols : 32;   // columns reduced at a time
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const CacheBars bar(smem + L::kBar);
  const CacheRanges ranges(smem + L::kRanges);
  volatile int* abort_flag = bar.abort_flag();
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) bar.init(128, 128);
  if (warp == 1) {
    tmem_alloc(bar.tmem_holder(), 256);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  griddep_launch_dependents();
  griddep_wait();  // lengths, queries and the new cache entries; the scratch of the call before
  tc_fence_before();
  ranges.find<kWork>(p, kWork * blockIdx.x, kWork * gridDim.x);
  tc_fence_after();
  const uint32_t tmem_base = *bar.tmem_holder();
  const bool no_loads = p.fault && blockIdx.x == 0;  // test hook: CTA 0's consumers wait out and abort

  // 64 columns take more registers than 384 threads can all have: 168 x 384 at launch = 88 x 128 +
  // 208 x 256
  if (warp < 4) {
    if constexpr (kCols == 64) setmaxnreg_dec<88>();
    if (warp == 0) {
      if (lane == 0 && !no_loads) produce_k<kWork>(p, ranges, bar, &tmK, smem + L::kK);
    } else if (warp == 3) {
      // rows of the product past the queries' box hold whatever was there: their columns are not used
      if (lane == 0 && !no_loads) produce_vq<kTwoWorkers>(p, ranges, bar, &tmQ, &tmV, smem, kCols, L::kQHalf, smem + L::kV);
    } else if (warp == 2) {
      clear_v<kWork>(p, ranges, bar, smem + L::kV);
    } else {
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, kN, 0, 0);   // K, Q both K-major
      constexpr uint32_t idesc_pv = idesc_bf16_f32(128, 64, 1, 1);  // V^T (d contiguous), P (rows contiguous)
      const uint32_t q_addr = smem_u32(smem), p_addr = smem_u32(smem + L::kP);
      const uint32_t k_addr = smem_u32(smem + L::kK), v_addr = smem_u32(smem + L::kV);
      issue_all<kTwoWorkers, 1>(
          p, ranges, bar,
          [&](int slot, int, int ks) {
            const uint64_t kd = sdesc_sw128(k_addr + ks * kKvTileBytes, 0, 1024);
            const uint64_t qd = sdesc_sw128(q_addr + slot * 2 * L::kQHalf, 0, 1024);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma_ss(tmem_base + slot * 64, kd + (((kk >> 2) * kKvHalfBytes + (kk & 3) * 32) >> 4),
                      qd + (((kk >> 2) * L::kQHalf + (kk & 3) * 32) >> 4), idesc_s, kk != 0);
          },
          [&](int slot, int, int vs, int, bool first) {
            const uint64_t vd = sdesc_sw128(v_addr + vs * kKvTileBytes, kKvHalfBytes, 1024);
            const uint64_t pd = sdesc_sw128(p_addr + slot * L::kPBytes, L::kPBytes, 1024);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)  // 16 keys: two groups of 8 rows of 128 bytes
              umma_ss(tmem_base + 128 + slot * 64, vd + ((kk * 2048) >> 4), pd + ((kk * 2048) >> 4), idesc_pv,
                      !(first && kk == 0));
          });
    }
  } else {
    if constexpr (kCols == 64) setmaxnreg_inc<208>();
    // ------------------------------------------------------------------ softmax
    const int slot = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;  // key of the tile; element d of O
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem_base + lane_off + slot * 64;
    const uint32_t t_o = tmem_base + lane_off + 128 + slot * 64;
    float* mu = reinterpret_cast<float*>(smem + L::kStats) + slot * 3 * 64;  // m, or 0 where m is -inf
    float* limit = mu + 64;                                                  // m + 8
    float* factor = mu + 128;
    uint8_t* P = smem + L::kP + slot * L::kPBytes;
    float* red = reinterpret_cast<float*>(P);  // [4 warps][kCols], while no P is in use
    const int bar_id = 1 + slot;
    const int worker = 2 * blockIdx.x + slot;
    const int units = p.n_kv;
    const int live_cols = 4 * p.T;
    // kCols columns of TMEM (at least 16 are read)
    auto load = [&](uint32_t at, uint32_t(&v)[kN]) {
      if constexpr (kN == 16) {
        tmem_ld16(at, v);
      } else {
#pragma unroll
        for (int c = 0; c < kN; c += 32) tmem_ld32(at + c, *reinterpret_cast<uint32_t(*)[32]>(&v[c]));
      }
      tmem_ld_wait();
    };
    // reduction of the slot's 128 threads, column by column, into red[warp][column]
    auto reduce = [&](const float* v, auto op) {
#pragma unroll
      for (int c = 0; c < kCols; c += kChunk) {
        float x[kChunk];
#pragma unroll
        for (int i = 0; i < kChunk; ++i) x[i] = v[c + i];
        const int col = reduce_columns<kChunk>(x, op);
        red[quarter * kCols + c + col] = x[0];
      }
    };
    KvWalk w = ranges.walk(slot, p);
    int flat = ranges.first_tile(slot);
    int items = 0, piece = 0;
    bool ok = true;
    for (; ok && !w.done(); w.next(units, p.n_new, p.S_max, [&](int b) { return __ldcg(p.kv_len + b); }), ++piece) {
      const int end = kv_end(w.len, p.n_new, p.S_max);
      const int safe = keys_all_see(p, w.len);
      float l[kCols];
#pragma unroll
      for (int i = 0; i < kCols; ++i) l[i] = 0.f;
      for (int j = 0; j < w.n; ++j, ++items) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar.s_full(slot), items & 1, abort_flag, p.status));
        // one decision for the slot's threads, which meet at the barriers below
        if (!(ok = named_bar_and(bar_id, 128, ok))) break;
        tc_fence_after();
        uint32_t sv[kN];
        load(t_s, sv);
        float s[kCols];
#pragma unroll
        for (int i = 0; i < kCols; ++i) s[i] = __uint_as_float(sv[i]);
        const int key0 = (w.first + j) * kKvTile;
        if (key0 + kKvTile > safe) {
          const int d = key0 + r - safe;  // drafted index of this thread's key
          if (d >= 0) {
            const bool in = end >= 0 && d < p.n_new;
            const int W = (p.T + 31) / 32;
            const uint32_t* m = p.mask ? p.mask + static_cast<size_t>(w.b) * p.T * W + (in ? d >> 5 : 0) : nullptr;
#pragma unroll
            for (int t = 0; t < kCols / 4; ++t) {
              const bool see = in && (!m || (t < p.T && ((__ldcg(m + t * W) >> (d & 31)) & 1u)));
              if (!see) s[4 * t] = s[4 * t + 1] = s[4 * t + 2] = s[4 * t + 3] = -INFINITY;
            }
          }
        }
        if constexpr (kScores) {  // raw scores of the four heads, for the weights (masked keys as -inf)
          reinterpret_cast<float4*>(p.scores)[static_cast<size_t>(flat + j) * kKvTile + r] =
              make_float4(s[0], s[1], s[2], s[3]);
          if (r == 0) p.tile_unit[flat + j] = make_int2(w.b * units + w.u, w.first + j);
        }
        bool over = j == 0;
        if (j > 0) {
#pragma unroll
          for (int i = 0; i < kCols; i += 4) {
            const float4 lim = *reinterpret_cast<const float4*>(limit + i);
            over |= s[i] * p.scale_log2 > lim.x || s[i + 1] * p.scale_log2 > lim.y || s[i + 2] * p.scale_log2 > lim.z ||
                    s[i + 3] * p.scale_log2 > lim.w;
          }
          over = !named_bar_and(bar_id, 128, !over);
        }
        if (over) {
          // P of the slot's last tile has been used up (its PV precedes this S)
          reduce(s, OpMax{});
          named_bar_sync(bar_id, 128);
          if (r < kCols) {
            const float top = fmaxf(fmaxf(red[r], red[kCols + r]), fmaxf(red[2 * kCols + r], red[3 * kCols + r]));
            const float old = j == 0 || limit[r] == -INFINITY ? -INFINITY : mu[r];
            const float m = fmaxf(old, top * p.scale_log2);
            factor[r] = m == -INFINITY ? 0.f : fast_exp2(old - m);
            mu[r] = m == -INFINITY ? 0.f : m;
            limit[r] = m + 8.f;
          }
          named_bar_sync(bar_id, 128);
          if (j > 0) {
            uint32_t o[kN];
            load(t_o, o);
#pragma unroll
            for (int i = 0; i < kCols; ++i) {
              l[i] *= factor[i];
              o[i] = __float_as_uint(__uint_as_float(o[i]) * factor[i]);
            }
            if constexpr (kN == 16) {
              tmem_st16(t_o, o);
            } else {
#pragma unroll
              for (int c = 0; c < kN; c += 32) tmem_st32(t_o + c, *reinterpret_cast<uint32_t(*)[32]>(&o[c]));
            }
            tmem_st_wait();
            tc_fence_before();
          }
        }
        // P as bf16 for the tensor product (the sum stays fp32): row r, 16-byte chunk c at c ^ (r & 7)
#pragma unroll
        for (int c = 0; c < (kCols + 7) / 8; ++c) {
          uint32_t pw[4];
#pragma unroll
          for (int i = 0; i < (kCols < 8 ? 2 : 4); ++i) {
            const int n = 8 * c + 2 * i;
            const float2 m2 = *reinterpret_cast<const float2*>(mu + n);
            const float a = fast_exp2(fmaf(s[n], p.scale_log2, -m2.x));
            const float b = fast_exp2(fmaf(s[n + 1], p.scale_log2, -m2.y));
            l[n] += a;
            l[n + 1] += b;
            pw[i] = pack_bf16x2(a, b);
          }
          uint8_t* dst = P + r * 128 + ((c ^ (r & 7)) << 4);
          if constexpr (kCols < 8)
            *reinterpret_cast<uint2*>(dst) = make_uint2(pw[0], pw[1]);
          else
            *reinterpret_cast<uint4*>(dst) = make_uint4(pw[0], pw[1], pw[2], pw[3]);
        }
        fence_proxy_async_smem();
        mbar_arrive(bar.p_lo(slot));
      }
      // ---------------------------------------------------------------- end of a piece
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar.o_full(slot), piece & 1, abort_flag, p.status));
      else break;  // every thread of the slot has left the loop at the same barrier
      if (!(ok = named_bar_and(bar_id, 128, ok))) break;
      tc_fence_after();
      uint32_t o[kN];
      load(t_o, o);
      tc_fence_before();
      mbar_arrive(bar.o_empty(slot));
      reduce(l, OpSum{});
      named_bar_sync(bar_id, 128);
      const bool whole = w.whole();
      const size_t ps = partial_slot(worker, w.first > 0);
      if (r < kCols) {
        const float sum = (red[r] + red[kCols + r]) + (red[2 * kCols + r] + red[3 * kCols + r]);
        const float m = limit[r] == -INFINITY ? -INFINITY : mu[r];
        // no visible key: zeros; a length out of range: NaN; a part of a unit stays as it is
        factor[r] = !whole ? 1.f : end < 0 ? __int_as_float(0x7FC00000) : (sum == 0.f ? 0.f : 1.f / sum);
        if (r < live_cols) {
          if (!whole) p.part_ml[ps * p.part_rows + r] = make_float2(m, sum);
          if (kScores && whole) p.unit_ml[(w.b * units + w.u) * 4 + r] = make_float2(m, sum);
        }
        if (r == 0 && w.first == 0) {
          if (kScores)
            p.unit_workers[w.b * units + w.u] =
                make_int2(worker, whole ? worker : range_owner(ranges.total(), ranges.workers(), flat + w.tiles - 1));
          if (end < 0) atomicOr(p.status, kDevErrRange);
        }
      }
      named_bar_sync(bar_id, 128);
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.h) + static_cast<size_t>(w.b) * p.T * (p.n_kv * 512) + w.u * 512 + r;
      float* part = p.part_o + ps * p.part_rows * 128 + r;
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        if (i < live_cols) {
          const float v = __uint_as_float(o[i]);
          if (whole)
            out[static_cast<size_t>(i >> 2) * (p.n_kv * 512) + (i & 3) * 128] = __float2bfloat16_rn(v * factor[i]);
          else
            part[i * 128] = v;
        }
      }
      flat += w.n;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 256);
  }
}

}  // namespace gqa
