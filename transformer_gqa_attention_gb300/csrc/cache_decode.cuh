// cache_decode.cuh — the decode attention that accumulates key weights: one position per sequence over
// caches whose lengths differ from sequence to sequence (cache_roles.cuh has the CTA's roles), handing
// its scores on to cache_weights_kernel.
//
// With the 4 rows (heads) of one position the products are turned round, so that the 128 keys of a
// tile fill the tensor core's rows and no lane idles for want of queries:
//   S^T = K Q^T    [128 keys, 4 heads]: one softmax thread per key, its four scores in registers,
//                  stored for the weights as one 16-byte piece
//   O^T = V^T P    [128 d, 4 heads]: V as stored (d contiguous), P [keys][heads] from shared memory
// The heads' maxima, which lie across threads here, are only needed to keep 2^(c s - m) in range: a
// tile whose scores all stay below m + 8 (one vote per tile) leaves m as it is; otherwise m is reduced
// across the slot's threads and O and l are rescaled.  l is kept per thread and summed once a piece.
// Each softmax slot is a worker with its own range of tiles.
// Bound by reading the cache: 64 sequences of 8192 keys (2.15 GB and 67 MB of scores written) in 338
// us, 6.55 TB/s.
//
// TMEM columns (64 each): S_0, S_1, O_0, O_1.
#pragma once

#include "cache_roles.cuh"

namespace gqa {

struct CacheDecodeSmem {
  static constexpr int kQHalf = 1024;           // 8 rows x 64 columns (4 heads, and rows that hold anything)
  static constexpr int kP = 8192;               // behind the slots' queries: N = 16 reads 16 rows
  static constexpr int kPBytes = 128 * 128;     // P: 128 keys x 64 columns (4 used), 128-byte swizzle
  static constexpr int kK = kP + 2 * kPBytes;
  static constexpr int kV = kK + kKStages * kKvTileBytes;
  static constexpr int kBar = kV + kVStages * kKvTileBytes;
  static constexpr int kRanges = kBar + CacheBars::kBytes;
  static constexpr int kStats = kRanges + CacheRanges::kBytes;  // per slot: [4 warps][4], then [4] m or 0, m + 8, factors
  static constexpr int kSlotStats = 32;                         // floats
  static constexpr int kBytes = kStats + 2 * kSlotStats * 4 + 1024;
};

__global__ void __launch_bounds__(384, 1)
    cache_decode_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const CacheAttnParams p) {
  using L = CacheDecodeSmem;
  constexpr int kWork = 2;
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
  // test hook: the last worker's CTA loads nothing, its consumers wait out and abort
  const bool no_loads = p.fault && static_cast<int>(blockIdx.x) == (ranges.workers() - 1) / kWork;

  if (warp == 0) {
    if (lane == 0 && !no_loads) produce_k<kWork>(p, ranges, bar, &tmK, smem + L::kK);
  } else if (warp == 3) {
    // rows of the product past the four heads hold whatever was there: their columns are not used
    if (lane == 0 && !no_loads) produce_vq<kTwoWorkers>(p, ranges, bar, &tmQ, &tmV, smem, 4, L::kQHalf, smem + L::kV);
  } else if (warp == 2) {
    clear_v<kWork>(p, ranges, bar, smem + L::kV);
  } else if (warp == 1) {
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, 16, 0, 0);   // K, Q both K-major
    constexpr uint32_t idesc_pv = idesc_bf16_f32(128, 64, 1, 1);  // V^T (d contiguous), P (heads contiguous)
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
  } else {
    // ------------------------------------------------------------------ softmax
    const int slot = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;  // key of the tile; element d of O
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem_base + lane_off + slot * 64;
    const uint32_t t_o = tmem_base + lane_off + 128 + slot * 64;
    float* red = reinterpret_cast<float*>(smem + L::kStats) + slot * L::kSlotStats;  // [4 warps][4 heads]
    float* mu = red + 16;      // m, or 0 where m is -inf
    float* limit = red + 20;   // m + 8
    float* factor = red + 24;
    uint8_t* P = smem + L::kP + slot * L::kPBytes + r * 128 + ((r & 7) << 4);  // row r, chunk 0 at 0 ^ (r & 7)
    const int bar_id = 1 + slot;
    const int worker = 2 * blockIdx.x + slot;
    const int units = p.n_kv;
    // four columns of TMEM (16 are read)
    auto load = [&](uint32_t at, float(&x)[4]) {
      uint32_t v[16];
      tmem_ld16(at, v);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(v[i]);
    };
    // the slot's 128 threads' values, head by head, into red[warp][head]
    auto reduce = [&](const float(&v)[4], auto op) {
      float x[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = op(x[i], __shfl_xor_sync(0xffffffffu, x[i], o));
      if (lane == 0) *reinterpret_cast<float4*>(red + 4 * quarter) = make_float4(x[0], x[1], x[2], x[3]);
    };
    KvWalk w = ranges.walk(slot, p);
    int items = 0, piece = 0;
    bool ok = true;
    for (; ok && !w.done(); w.next(units, p.n_new, p.S_max, [&](int b) { return __ldcg(p.kv_len + b); }), ++piece) {
      const int end = kv_end(w.len, p.n_new, p.S_max);  // (out of range: -1, no key is visible)
      const int flat = w.tile(w.first, units);
      int4 unit;  // of the weights kernel's tile records
      if (r == 0)
        unit = make_int4(w.b * units + w.u, w.first, range_owner(ranges.total(), ranges.workers(), w.place(0)),
                         range_owner(ranges.total(), ranges.workers(), w.place(w.tiles - 1)));
      float l[4] = {0.f, 0.f, 0.f, 0.f};
      for (int j = 0; j < w.n; ++j, ++items) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar.s_full(slot), items & 1, abort_flag, p.status));
        tc_fence_after();
        float s[4];
        load(t_s, s);
        if ((w.first + j) * kKvTile + r >= end) s[0] = s[1] = s[2] = s[3] = -INFINITY;
        reinterpret_cast<float4*>(p.scores)[static_cast<size_t>(flat + j) * kKvTile + r] = make_float4(s[0], s[1], s[2], s[3]);
        if (r == 0) p.tile_unit[flat + j] = make_int4(unit.x, unit.y + j, unit.z, unit.w);
        bool over = j == 0;
        if (j > 0) {
          const float4 lim = *reinterpret_cast<const float4*>(limit);
          over = s[0] * p.scale_log2 > lim.x || s[1] * p.scale_log2 > lim.y || s[2] * p.scale_log2 > lim.z ||
                 s[3] * p.scale_log2 > lim.w;
        }
        // one decision for the slot's threads: a maximum has grown, or a wait was given up
        if (!named_bar_and(bar_id, 128, ok && !over)) {
          if (!(ok = named_bar_and(bar_id, 128, ok))) break;
          reduce(s, [](float a, float b) { return fmaxf(a, b); });
          named_bar_sync(bar_id, 128);
          if (r < 4) {
            const float top = fmaxf(fmaxf(red[r], red[4 + r]), fmaxf(red[8 + r], red[12 + r]));
            const float old = j == 0 || limit[r] == -INFINITY ? -INFINITY : mu[r];
            const float m = fmaxf(old, top * p.scale_log2);
            factor[r] = m == -INFINITY ? 0.f : fast_exp2(old - m);
            mu[r] = m == -INFINITY ? 0.f : m;
            limit[r] = m + 8.f;
          }
          named_bar_sync(bar_id, 128);
          if (j > 0) {  // O holds the sum through the slot's tile before (its PV precedes this S)
            uint32_t o[16];
            tmem_ld16(t_o, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              l[i] *= factor[i];
              o[i] = __float_as_uint(__uint_as_float(o[i]) * factor[i]);
            }
            tmem_st16(t_o, o);
            tmem_st_wait();
          }
        }
        const float4 m4 = *reinterpret_cast<const float4*>(mu);
        const float e[4] = {fast_exp2(fmaf(s[0], p.scale_log2, -m4.x)), fast_exp2(fmaf(s[1], p.scale_log2, -m4.y)),
                            fast_exp2(fmaf(s[2], p.scale_log2, -m4.z)), fast_exp2(fmaf(s[3], p.scale_log2, -m4.w))};
#pragma unroll
        for (int i = 0; i < 4; ++i) l[i] += e[i];
        // P as bf16 for the tensor product (the sum stays fp32)
        *reinterpret_cast<uint2*>(P) = make_uint2(pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]));
        fence_proxy_async_smem();
        // this arrival lets the issuer write the next tile's scores over the ones read above, and add to O
        tc_fence_before();
        mbar_arrive(bar.p_lo(slot));
      }
      // ---------------------------------------------------------------- end of a piece
      if (!ok) break;  // every thread of the slot has left the tiles at the same barrier
      ok = __all_sync(0xffffffffu, mbar_wait(bar.o_full(slot), piece & 1, abort_flag, p.status));
      if (!(ok = named_bar_and(bar_id, 128, ok))) break;
      tc_fence_after();
      float o[4];
      load(t_o, o);
      tc_fence_before();
      mbar_arrive(bar.o_empty(slot));
      reduce(l, [](float a, float b) { return a + b; });
      named_bar_sync(bar_id, 128);
      const bool whole = w.whole();
      const size_t ps = partial_slot(worker, w.first > 0);
      if (r < 4) {
        const float sum = (red[r] + red[4 + r]) + (red[8 + r] + red[12 + r]);
        const float m = limit[r] == -INFINITY ? -INFINITY : mu[r];
        // no visible key: zeros; a length out of range: NaN; a part of a unit stays as it is
        factor[r] = !whole ? 1.f : end < 0 ? __int_as_float(0x7FC00000) : (sum == 0.f ? 0.f : 1.f / sum);
        if (whole)
          p.unit_ml[(w.b * units + w.u) * 4 + r] = make_float2(m, sum);
        else
          p.part_ml[ps * p.part_rows + r] = make_float2(m, sum);
        if (r == 0 && w.first == 0 && end < 0) atomicOr(p.status, kDevErrRange);
      }
      named_bar_sync(bar_id, 128);
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.h) + static_cast<size_t>(w.b) * (p.n_kv * 512) + w.u * 512 + r;
      float* part = p.part_o + ps * p.part_rows * 128 + r;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (whole)
          out[i * 128] = __float2bfloat16_rn(o[i] * factor[i]);
        else
          part[i * 128] = o[i];
      }
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
