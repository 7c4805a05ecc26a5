// cache_attn.cuh — attention of 17 and more positions per sequence over caches whose lengths differ
// from sequence to sequence (cache_roles.cuh has the CTA's roles; cache_attn_few.cuh the kernel for
// fewer positions), and the kernels that finish either one's work.
//
// The four query heads of a kv head read the same keys and values, so the tensor core's 128 rows
// are 32 positions x 4 heads: row 4t + h.  Every K/V byte then serves all rows of up to 32 (or,
// with two row tiles, 64) positions: 4 T rows do 4 T x 128 x 4 FLOP per key of 512 bytes.
//   S = Q K^T into TMEM, softmax, P over S in TMEM, O += P V.
// A piece that is a whole unit is normalised and stored to h; another leaves an unnormalised O
// (fp32) with its maximum and sum in the scratch, which cache_merge_kernel joins.
//
// TMEM columns: S_0/P_0 at 0, S_1/P_1 at 128, O_0 at 256, O_1 at 384.
#pragma once

#include "cache_roles.cuh"

namespace gqa {

struct CacheAttnSmem {
  static constexpr int kK = 2 * kKvTileBytes;  // behind two query tiles
  static constexpr int kV = kK + kKStages * kKvTileBytes;
  static constexpr int kBar = kV + kVStages * kKvTileBytes;
  static constexpr int kRanges = kBar + CacheBars::kBytes;
  static constexpr int kHalves = kRanges + CacheRanges::kBytes;  // [2 halves][128 rows] floats exchanged
  static constexpr int kBytes = kHalves + 2 * 128 * 4 + 1024;
};

// kOneTile: two threads share a row, warps 4..7 keys 0..63 of a tile, warps 8..11 keys 64..127 (TMEM
// lanes belong to a warp's number mod 4), which halves the time between a tile's S and its PV.  The
// row maximum is only needed to keep 2^(c s - m) in range: m follows the scores when one of them
// passes m + 8, on a vote of the 64 threads of a row group; then the two halves' maxima are exchanged
// and O and l rescaled.
__device__ __forceinline__ void softmax_halves(const CacheAttnParams& p, const CacheRanges& ranges, const CacheBars& bar,
                                               uint32_t tmem_base, float* exchange) {
  constexpr int kMode = kOneTile, kItems = 1;
  volatile int* abort_flag = bar.abort_flag();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = (warp - 4) >> 2;  // keys 64 half .. + 63; columns 64 half .. + 63 of O
  const int quarter = warp & 3;
  const int r = quarter * 32 + lane;  // row of the tile: position r / 4, head r & 3
  const int bar_id = 1 + quarter;     // the two warps of a row group
  const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
  float* mine = exchange + half * 128 + r;
  const float* other = exchange + (half ^ 1) * 128 + r;
  const int W = (p.T + 31) / 32;
  const int units = p.n_kv * p.row_groups;
  KvWalk w = ranges.walk(0, p);
  int it = 0, piece = 0;
  bool ok = true;
  for (; ok && !w.done(); w.next(units, p.n_new, p.S_max, [&](int b) { return __ldcg(p.kv_len + b); }), ++piece) {
    const int end = kv_end(w.len, p.n_new, p.S_max);
    const int safe = keys_all_see(p, w.len);
    const int g = w.u / p.row_groups;
    const int t0 = (w.u - g * p.row_groups) * p.group_pos;
    float m_used[kItems], l_sum[kItems];
    for (int j = 0; ok && j < w.n; ++j, ++it) {
      const int key0 = (w.first + j) * kKvTile + 64 * half;
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const int slot = kMode == kOneTile ? it & 1 : i;
        const int turn = kMode == kOneTile ? it >> 1 : it;
        const uint32_t t_s = t_row + slot * 128;
        const bool warp_live = t0 + 32 * i + quarter * 8 < p.T;
        ok = __all_sync(0xffffffffu, mbar_wait(bar.s_full(slot), turn & 1, abort_flag, p.status));
        if (!warp_live) {  // rows past the last position: whatever their P is, their O is not used
          if (!ok) break;
          mbar_arrive(half ? bar.p_hi(slot) : bar.p_lo(slot));
          continue;
        }
        tc_fence_after();
        uint32_t sv[64];
        tmem_ld32(t_s + 64 * half, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
        tmem_ld32(t_s + 64 * half + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
        tmem_ld_wait();
        if (key0 + 64 > safe) {
          const int t = t0 + 32 * i + (r >> 2);
          const bool live = t < p.T;
          const uint32_t* mask = p.mask ? p.mask + (static_cast<size_t>(w.b) * p.T + (live ? t : 0)) * W : nullptr;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t bits = key_bits(mask, W, end < 0 ? 0 : p.n_new, key0 + 32 * c - safe, live);
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!((bits >> k) & 1u)) sv[32 * c + k] = 0xFF800000u;  // -inf
          }
        }
        float m8[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) m8[k] = __uint_as_float(sv[k]);
#pragma unroll
        for (int k = 0; k < 28; ++k)
          m8[k & 7] = max3f(m8[k & 7], __uint_as_float(sv[8 + 2 * k]), __uint_as_float(sv[9 + 2 * k]));
        const float mx = max3f(max3f(m8[0], m8[1], m8[2]), max3f(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
        const float m_half = mx * p.scale_log2;
        // One decision for the row group's 64 threads: a row's maximum has grown (or this is its first
        // tile), or a wait was given up, which ends the walk of both warps here.  Past the barrier both
        // halves of S have been read, and P may take their place.
        const bool over = j == 0 || m_half > m_used[i] + 8.0f;
        tc_fence_before();
        if (!named_bar_and(bar_id, 64, ok && !over)) {
          if (!(ok = named_bar_and(bar_id, 64, ok))) break;
          *mine = m_half;
          named_bar_sync(bar_id, 64);
          const float m_old = j == 0 ? -INFINITY : m_used[i];
          const float m_new = fmaxf(m_old, fmaxf(m_half, *other));
          const float alpha = m_new == -INFINITY ? 0.f : fast_exp2(m_old - m_new);
          m_used[i] = m_new;
          l_sum[i] = j == 0 ? 0.f : l_sum[i] * alpha;
          if (j > 0) {  // this half's columns of O, which holds the sum through the tile before
            const uint32_t t_o = t_row + 256 + 128 * piece_buffer<kMode>(0, i, piece) + 64 * half;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t v[32];
              tmem_ld32(t_o + c * 32, v);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha);
              tmem_st32(t_o + c * 32, v);
            }
            tmem_st_wait();
            tc_fence_before();
          }
          named_bar_sync(bar_id, 64);  // both halves of O are rescaled before either half of P is released
        }
        tc_fence_after();
        const float mu = (m_used[i] == -INFINITY) ? 0.f : m_used[i];
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
        const float2 nmu2 = make_float2(-mu, -mu);
        float2 l4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pw[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 a = ffma2(make_float2(__uint_as_float(sv[c * 32 + 2 * e]), __uint_as_float(sv[c * 32 + 2 * e + 1])),
                                   sc2, nmu2);
            const float2 pe = make_float2(fast_exp2(a.x), fast_exp2(a.y));
            l4[e & 3] = fadd2(l4[e & 3], pe);
            pw[e] = pack_bf16x2(pe.x, pe.y);  // P feeds a bf16 tensor product; the sum stays fp32
          }
          tmem_st16(t_s + 32 * half + c * 16, pw);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(half ? bar.p_hi(slot) : bar.p_lo(slot));
        const float2 l2 = fadd2(fadd2(l4[0], l4[1]), fadd2(l4[2], l4[3]));
        l_sum[i] += l2.x + l2.y;
      }
    }
    // ---------------------------------------------------------------- end of a piece
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int at = piece_buffer<kMode>(0, i, piece);
      const bool warp_live = t0 + 32 * i + quarter * 8 < p.T;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar.o_full(at), piece_turn<kMode>(piece) & 1, abort_flag, p.status));
      if (!warp_live) {
        if (!ok) break;
        mbar_arrive(bar.o_empty(at));
        continue;
      }
      if (!(ok = named_bar_and(bar_id, 64, ok))) break;
      tc_fence_after();
      uint32_t v[64];
      const uint32_t t_o = t_row + 256 + 128 * at + 64 * half;
      tmem_ld32(t_o, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
      tmem_ld32(t_o + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
      *mine = l_sum[i];
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(bar.o_empty(at));
      named_bar_sync(bar_id, 64);
      const float o_sum = *other;
      const float l = half ? o_sum + l_sum[i] : l_sum[i] + o_sum;
      named_bar_sync(bar_id, 64);  // read before the next exchange
      const int t = t0 + 32 * i + (r >> 2);
      if (t < p.T) {
        if (w.whole()) {
          // no visible key: zeros; a length out of range: NaN
          const float inv = end < 0 ? __int_as_float(0x7FC00000) : (l == 0.f ? 0.f : 1.f / l);
          uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.h) +
                                                (static_cast<size_t>(w.b) * p.T + t) * (p.n_kv * 512) +
                                                (g * 4 + (r & 3)) * 128 + 64 * half);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            out[k] = make_uint4(pack_bf16x2(__uint_as_float(v[8 * k + 0]) * inv, __uint_as_float(v[8 * k + 1]) * inv),
                                pack_bf16x2(__uint_as_float(v[8 * k + 2]) * inv, __uint_as_float(v[8 * k + 3]) * inv),
                                pack_bf16x2(__uint_as_float(v[8 * k + 4]) * inv, __uint_as_float(v[8 * k + 5]) * inv),
                                pack_bf16x2(__uint_as_float(v[8 * k + 6]) * inv, __uint_as_float(v[8 * k + 7]) * inv));
        } else {
          const int row = 128 * i + r;
          const size_t ps = partial_slot(blockIdx.x, w.first > 0);
          float4* part = reinterpret_cast<float4*>(p.part_o) + (ps * 32 + 16 * half) * p.part_rows + row;
#pragma unroll
          for (int k = 0; k < 16; ++k)
            part[k * p.part_rows] = make_float4(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1]),
                                                __uint_as_float(v[4 * k + 2]), __uint_as_float(v[4 * k + 3]));
          if (half == 0) p.part_ml[ps * p.part_rows + row] = make_float2(m_used[i], l);
        }
        if (i == 0 && r == 0 && half == 0 && w.first == 0 && end < 0) atomicOr(p.status, kDevErrRange);
      }
    }
  }
}

// kTwoTiles: warps 4..7 have row tile 0, warps 8..11 row tile 1, a thread a row, so that the row
// tiles' softmaxes run side by side, each under the other's S and PV.
__device__ __forceinline__ void softmax_rows(const CacheAttnParams& p, const CacheRanges& ranges, const CacheBars& bar,
                                             uint32_t tmem_base) {
  volatile int* abort_flag = bar.abort_flag();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slot = (warp - 4) >> 2;
  const int quarter = warp & 3;
  const int r = quarter * 32 + lane;  // row of the tile: position r / 4, head r & 3
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t t_s = tmem_base + lane_off + slot * 128;
  const uint32_t t_o = tmem_base + lane_off + 256 + slot * 128;
  KvWalk w = ranges.walk(0, p);
  const int units = p.n_kv * p.row_groups;
  int items = 0, piece = 0;
  bool ok = true;
  // first position of the slot's rows
  auto first_pos = [&](int u) { return u % p.row_groups * p.group_pos + 32 * slot; };
  for (; ok && !w.done(); w.next(units, p.n_new, p.S_max, [&](int b) { return __ldcg(p.kv_len + b); }), ++piece) {
    const bool warp_live = first_pos(w.u) + quarter * 8 < p.T;
    const int safe = keys_all_see(p, w.len);
    int key0 = w.first * kKvTile;
    float m_used = -INFINITY;
    float l_sum = 0.f;
    for (int j = 0; j < w.n; ++j, ++items, key0 += kKvTile) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar.s_full(slot), items & 1, abort_flag, p.status));
      if (!ok) break;
      if (!warp_live) {  // rows past the last position: whatever their P is, their O is not used
        mbar_arrive(bar.p_lo(slot));
        mbar_arrive(bar.p_hi(slot));
        continue;
      }
      tc_fence_after();
      uint32_t sv[128];
      tmem_ld32(t_s + 0, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
      tmem_ld32(t_s + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
      tmem_ld32(t_s + 64, *reinterpret_cast<uint32_t(*)[32]>(&sv[64]));
      tmem_ld32(t_s + 96, *reinterpret_cast<uint32_t(*)[32]>(&sv[96]));
      tmem_ld_wait();
      if (key0 + kKvTile > safe) {
        const int n_new = kv_end(w.len, p.n_new, p.S_max) < 0 ? 0 : p.n_new;
        const int t = first_pos(w.u) + (r >> 2);
        const int W = (p.T + 31) / 32;
        const bool live = t < p.T;
        const uint32_t* mask = p.mask ? p.mask + (static_cast<size_t>(w.b) * p.T + (live ? t : 0)) * W : nullptr;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t bits = key_bits(mask, W, n_new, key0 + 32 * i - safe, live);
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (!((bits >> k) & 1u)) sv[32 * i + k] = 0xFF800000u;  // -inf
        }
      }
      float m8[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) m8[i] = __uint_as_float(sv[i]);
#pragma unroll
      for (int k = 0; k < 60; ++k)
        m8[k & 7] = max3f(m8[k & 7], __uint_as_float(sv[8 + 2 * k]), __uint_as_float(sv[9 + 2 * k]));
      const float mx = max3f(max3f(m8[0], m8[1], m8[2]), max3f(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
      const float m_tile = mx * p.scale_log2;
      // lazy rescale: O and l follow the maximum only when it grows by more than 2^8
      float alpha = 1.f;
      bool grow = false;
      if (j == 0) {
        m_used = m_tile;
      } else if (m_tile > m_used + 8.0f) {
        grow = true;
        alpha = fast_exp2(m_used - m_tile);
        l_sum *= alpha;
        m_used = m_tile;
      }
      const float mu = (m_used == -INFINITY) ? 0.f : m_used;
      const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
      const float2 nmu2 = make_float2(-mu, -mu);
      float2 l4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
        for (int c = 2 * hf; c < 2 * hf + 2; ++c) {
          uint32_t pw[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 a = ffma2(make_float2(__uint_as_float(sv[c * 32 + 2 * e]), __uint_as_float(sv[c * 32 + 2 * e + 1])),
                                   sc2, nmu2);
            const float2 pe = make_float2(fast_exp2(a.x), fast_exp2(a.y));
            l4[e & 3] = fadd2(l4[e & 3], pe);
            pw[e] = pack_bf16x2(pe.x, pe.y);  // P feeds a bf16 tensor product; the sum stays fp32
          }
          tmem_st16(t_s + c * 16, pw);
        }
        if (hf == 0 && __any_sync(0xffffffffu, grow)) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            tmem_ld32(t_o + c * 32, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
            tmem_st32(t_o + c * 32, v);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(hf == 0 ? bar.p_lo(slot) : bar.p_hi(slot));
      }
      const float2 l2 = fadd2(fadd2(l4[0], l4[1]), fadd2(l4[2], l4[3]));
      l_sum += l2.x + l2.y;
    }
    // ---------------------------------------------------------------- end of a piece
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar.o_full(slot), piece & 1, abort_flag, p.status));
    if (!ok) break;
    tc_fence_after();
    if (!warp_live) {
      mbar_arrive(bar.o_empty(slot));
    } else {
      uint32_t v[128];
      tmem_ld32(t_o + 0, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
      tmem_ld32(t_o + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
      tmem_ld32(t_o + 64, *reinterpret_cast<uint32_t(*)[32]>(&v[64]));
      tmem_ld32(t_o + 96, *reinterpret_cast<uint32_t(*)[32]>(&v[96]));
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(bar.o_empty(slot));
      const int g = w.u / p.row_groups;
      const int t = first_pos(w.u) + (r >> 2);
      const int end = kv_end(w.len, p.n_new, p.S_max);
      if (t < p.T) {
        const int row = 128 * slot + r;
        if (w.whole()) {
          // no visible key: zeros; a length out of range: NaN
          const float inv = end < 0 ? __int_as_float(0x7FC00000) : (l_sum == 0.f ? 0.f : 1.f / l_sum);
          uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.h) +
                                                (static_cast<size_t>(w.b) * p.T + t) * (p.n_kv * 512) +
                                                (g * 4 + (r & 3)) * 128);
#pragma unroll
          for (int k = 0; k < 16; ++k)
            out[k] = make_uint4(pack_bf16x2(__uint_as_float(v[8 * k + 0]) * inv, __uint_as_float(v[8 * k + 1]) * inv),
                                pack_bf16x2(__uint_as_float(v[8 * k + 2]) * inv, __uint_as_float(v[8 * k + 3]) * inv),
                                pack_bf16x2(__uint_as_float(v[8 * k + 4]) * inv, __uint_as_float(v[8 * k + 5]) * inv),
                                pack_bf16x2(__uint_as_float(v[8 * k + 6]) * inv, __uint_as_float(v[8 * k + 7]) * inv));
        } else {
          const size_t ps = partial_slot(blockIdx.x, w.first > 0);
          float4* part = reinterpret_cast<float4*>(p.part_o) + ps * 32 * p.part_rows + row;
#pragma unroll
          for (int k = 0; k < 32; ++k)
            part[k * p.part_rows] = make_float4(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1]),
                                                __uint_as_float(v[4 * k + 2]), __uint_as_float(v[4 * k + 3]));
          p.part_ml[ps * p.part_rows + row] = make_float2(m_used, l_sum);
        }
        if (r == 0 && w.first == 0 && end < 0) atomicOr(p.status, kDevErrRange);
      }
    }
  }
}

// kMode: kOneTile (at most 32 positions) or kTwoTiles (groups of 64).
template <int kMode>
__global__ void __launch_bounds__(384, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const CacheAttnParams p) {
  using L = CacheAttnSmem;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const CacheBars bar(smem + L::kBar);
  const CacheRanges ranges(smem + L::kRanges);
  volatile int* abort_flag = bar.abort_flag();
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) bar.init(kMode == kTwoTiles ? 128 : 256);
  if (warp == 1) {
    tmem_alloc(bar.tmem_holder(), 512);
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
  ranges.find<1>(p);
  tc_fence_after();
  const uint32_t tmem_base = *bar.tmem_holder();
  const bool no_loads = p.fault && blockIdx.x == 0;  // test hook: CTA 0's consumers wait out and abort

  // kTwoTiles: a row of 128 scores per thread takes more registers than 384 threads can all have:
  // 168 x 384 at launch = 88 x 128 + 208 x 256
  if (warp < 4) {
    if constexpr (kMode == kTwoTiles) setmaxnreg_dec<88>();
    if (warp == 0) {
      if (lane == 0 && !no_loads) produce_k<1>(p, ranges, bar, &tmK, smem + L::kK);
    } else if (warp == 3) {
      if (lane == 0 && !no_loads) produce_vq<kMode>(p, ranges, bar, &tmQ, &tmV, smem, 128, kKvHalfBytes, smem + L::kV);
    } else if (warp == 2) {
      clear_v<1>(p, ranges, bar, smem + L::kV);
    } else {
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, 0, 0);   // Q, K both K-major
      constexpr uint32_t idesc_pv = idesc_bf16_f32(128, 128, 0, 1);  // P (TMEM), V MN-major
      const uint32_t q_addr = smem_u32(smem), k_addr = smem_u32(smem + L::kK), v_addr = smem_u32(smem + L::kV);
      issue_all<kMode, 2>(
          p, ranges, bar,
          [&](int slot, int q, int ks) {
            const uint64_t qd = sdesc_sw128(q_addr + q * kKvTileBytes, 0, 1024);
            const uint64_t kd = sdesc_sw128(k_addr + ks * kKvTileBytes, 0, 1024);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t off = ((kk >> 2) * kKvHalfBytes + (kk & 3) * 32) >> 4;  // descriptor address units
              umma_ss(tmem_base + slot * 128, qd + off, kd + off, idesc_s, kk != 0);
            }
          },
          [&](int slot, int o, int vs, int hf, bool first) {
            const uint64_t vd = sdesc_sw128(v_addr + vs * kKvTileBytes, kKvHalfBytes, 1024);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int kk = 4 * hf + i;
              umma_ts(tmem_base + 256 + o * 128, tmem_base + slot * 128 + kk * 8, vd + ((kk * 2048) >> 4), idesc_pv,
                      !(first && kk == 0));
            }
          });
    }
  } else if constexpr (kMode == kTwoTiles) {
    setmaxnreg_inc<208>();
    softmax_rows(p, ranges, bar, tmem_base);
  } else {
    softmax_halves(p, ranges, bar, tmem_base, reinterpret_cast<float*>(smem + L::kHalves));
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// Unnormalised sum of pieces k0, k0 + step, ... of a block of a cut unit's O, N float4 per lane:
// with kByRow (scratch [row][128 d], at most kFewPos positions) rows row0 .. row0 + rows - 1 (at
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

constexpr int kMergeY = 8;      // blocks per worker
constexpr int kMergeFewY = 4;   // at most kFewPos positions

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

template <bool kByRow>
__global__ void __launch_bounds__(256) cache_merge_kernel(const CacheAttnParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int v = blockIdx.x;
  const int4 d = __ldcg(p.merge + v);
  const int st = *reinterpret_cast<volatile const int*>(p.status);
  // after a wait that ran out the scratch may be unwritten
  if (d.x < 0 || (st & kDevErrTimeout)) return;
  merge_unit<kByRow>(p, d, (v - d.z) * gridDim.y + blockIdx.y, (d.w - d.z) * gridDim.y);
}

// The decode step with key weights: blocks 0 .. workers - 1 merge, the others add each key's
// weight, the sum over the four heads of 2^(c s - M) / l, to the running sums, one key tile per warp
// at a time.
__global__ void __launch_bounds__(256) cache_weights_kernel(const CacheAttnParams p, int workers) {
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
  // tiles of a warp are n_warps apart: neighbouring warps read neighbouring scores
  for (int i = (blockIdx.x - workers) * 8 + warp; i < total; i += n_warps) {
    const int2 tu = __ldcg(p.tile_unit + i);
    const float4* s = reinterpret_cast<const float4*>(p.scores) + static_cast<size_t>(i) * kKvTile;
    float x[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 v = __ldcg(s + 32 * k + lane);
      x[0][k] = v.x;
      x[1][k] = v.y;
      x[2][k] = v.z;
      x[3][k] = v.w;
    }
    const int2 cs = __ldcg(p.unit_workers + tu.x);
    float* w = p.weights + static_cast<size_t>(tu.x) * p.S_max + tu.y * kKvTile;
    bool seen[4];
    float a[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // -inf in all four heads: past the end (or of no weight)
      seen[k] = x[0][k] != -INFINITY || x[1][k] != -INFINITY || x[2][k] != -INFINITY || x[3][k] != -INFINITY;
      a[k] = seen[k] ? __ldcg(w + 32 * k + lane) : 0.f;
    }
    float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      float2 m = make_float2(-INFINITY, 0.f);
      if (cs.x == cs.y) {
        m = __ldcg(p.unit_ml + tu.x * 4 + h);
      } else {  // a cut unit: its pieces' maxima and sums, shared by the lanes
        for (int k = lane; k <= cs.y - cs.x; k += 32) {
          const int ps = k ? partial_slot(cs.x + k, true) : partial_slot(cs.x, false);
          const float2 o = __ldcg(p.part_ml + static_cast<size_t>(ps) * R + h);
          const float top = fmaxf(m.x, o.x), tz = top == -INFINITY ? 0.f : top;
          m = make_float2(top, m.y * fast_exp2(m.x - tz) + o.y * fast_exp2(o.x - tz));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const float2 q = make_float2(__shfl_xor_sync(0xffffffffu, m.x, o), __shfl_xor_sync(0xffffffffu, m.y, o));
          const float top = fmaxf(m.x, q.x), tz = top == -INFINITY ? 0.f : top;
          m = make_float2(top, m.y * fast_exp2(m.x - tz) + q.y * fast_exp2(q.x - tz));
        }
      }
      const float M = m.x == -INFINITY ? 0.f : m.x;
      const float inv = 1.f / m.y;
#pragma unroll
      for (int k = 0; k < 4; ++k) add[k] += fast_exp2(fmaf(x[h][k], p.scale_log2, -M)) * inv;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (seen[k]) w[32 * k + lane] = a[k] + add[k];
  }
}

}  // namespace gqa
