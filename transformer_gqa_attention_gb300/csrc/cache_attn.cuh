// cache_attn.cuh — attention of up to 32 positions per sequence over caches whose lengths differ from
// sequence to sequence (cache_roles.cuh has the CTA's roles; cache_attn_pair.cuh the kernel for more).
//
// The four query heads of a kv head read the same keys and values, so the tensor core's 128 rows
// are 32 positions x 4 heads: row 4t + h.  Every K/V byte then serves all rows of up to 32
// positions: 4 T rows do 4 T x 128 x 4 FLOP per key of 512 bytes, far below what the tensor cores could
// do, so reading the keys and values bounds it: 32 sequences of 4000 keys (528 MB) take 88 us with 8
// tokens (6.0 TB/s) and 95 with 32, with the merge; 8 ragged ones of up to 4000 keys and 26 tokens (73 MB)
// 23.5, of which the merge is 3 and a CTA's first tile 5; one of 300 keys and 8 tokens 9.1, all latency.
// Keys on the tensor core's rows, as the decode step has them (cache_decode.cuh): 106 us for 8 tokens
// where this takes 87.
//   S = Q K^T into TMEM, softmax, P over S in TMEM, O += P V.
// S alternates between two buffers from tile to tile, queries and O from unit to unit, so that the end
// of one unit (last PV, normalisation, stores) passes under the next one's first tiles.
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
  static constexpr int kExchange = kRanges + CacheRanges::kBytes;  // [2 halves][128 rows] floats
  static constexpr int kBytes = kExchange + 2 * 128 * 4 + 1024;
};

// Groups of eight lanes with eight pieces each: lane j gets piece j of every lane, x[k] from lane k.
__device__ __forceinline__ void transpose8(uint4 (&x)[8]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 4; d > 0; d >>= 1) {
    const bool up = lane & d;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k & d) continue;
      const uint4 give = up ? x[k] : x[k + d];
      const uint4 got = make_uint4(__shfl_xor_sync(0xffffffffu, give.x, d), __shfl_xor_sync(0xffffffffu, give.y, d),
                                   __shfl_xor_sync(0xffffffffu, give.z, d), __shfl_xor_sync(0xffffffffu, give.w, d));
      x[k] = up ? got : x[k];
      x[k + d] = up ? x[k + d] : got;
    }
  }
}

// The end of a piece for a row's thread, which has columns 64 half .. + 63 of O, unnormalised, in v: a whole
// unit goes to h, another into the scratch.  Called by whole warps; row tile `tile` of the worker's.
__device__ __forceinline__ void store_piece(const CacheAttnParams& p, const KvWalk& w, int end, int g, int t0, int tile,
                                            int worker, int half, int quarter, float m, float l, const uint32_t (&v)[64]) {
  const int lane = threadIdx.x & 31;
  auto value = [&](int i) { return __uint_as_float(v[i]); };
  if (w.whole()) {
    // no visible key: zeros; a length out of range: NaN
    const float inv = end < 0 ? __int_as_float(0x7FC00000) : (l == 0.f ? 0.f : 1.f / l);
    uint4 o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      o[k] = make_uint4(pack_bf16x2(value(8 * k) * inv, value(8 * k + 1) * inv),
                        pack_bf16x2(value(8 * k + 2) * inv, value(8 * k + 3) * inv),
                        pack_bf16x2(value(8 * k + 4) * inv, value(8 * k + 5) * inv),
                        pack_bf16x2(value(8 * k + 6) * inv, value(8 * k + 7) * inv));
    // A lane has 128 bytes of its row; eight lanes exchange theirs, so that they store one row at a time
    // (each lane its own row would be 32 pieces of 16 bytes an instruction).
    transpose8(o);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int row = quarter * 32 + (lane & 24) + k, t = t0 + (row >> 2);
      if (t < p.T)
        reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.h) +
                                 (static_cast<size_t>(w.b) * p.T + t) * (p.n_kv * 512) + (g * 4 + (row & 3)) * 128 +
                                 64 * half)[lane & 7] = o[k];
    }
  } else if (t0 + quarter * 8 + (lane >> 2) < p.T) {
    const int row = 128 * tile + quarter * 32 + lane;
    const size_t ps = partial_slot(worker, w.first > 0);
    float4* part = reinterpret_cast<float4*>(p.part_o) + (ps * 32 + 16 * half) * p.part_rows + row;
#pragma unroll
    for (int k = 0; k < 16; ++k)
      part[k * p.part_rows] = make_float4(value(4 * k), value(4 * k + 1), value(4 * k + 2), value(4 * k + 3));
    if (half == 0) p.part_ml[ps * p.part_rows + row] = make_float2(m, l);
  }
  if (tile == 0 && quarter == 0 && lane == 0 && half == 0 && w.first == 0 && end < 0) atomicOr(p.status, kDevErrRange);
}

// The softmax warps (warps 4..11), whose rows are positions t0 .. t0 + 31 of a unit.  Two threads share a row: warps 4..7 take keys 0..63 of a key tile, warps 8..11 keys 64..127
// (TMEM lanes belong to a warp's number mod 4), which halves the time between a tile's S and its PV.
// The row maximum is only needed to keep 2^(c s - m) in range: m follows the scores when one of them
// passes m + 8, on a vote of the 64 threads of a row group; then the two halves' maxima are exchanged
// and O and l rescaled.
__device__ __forceinline__ void softmax_halves(const CacheAttnParams& p, const CacheRanges& ranges, const CacheBars& bar,
                                               uint32_t tmem_base, float* exchange) {
  constexpr int kS = 2, kO = 2;  // buffers of S and O
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
  volatile int* abort_flag = bar.abort_flag();
  auto wait = [&](uint64_t* b, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(b, parity, abort_flag, p.status));
  };
  auto arrive_p = [&](int slot) { mbar_arrive(half ? bar.p_hi(slot) : bar.p_lo(slot)); };
  KvWalk w = ranges.walk(0, p);
  int it = 0, piece = 0;
  bool ok = true;
  for (; ok && !w.done(); w.next(units, p.n_new, p.S_max, [&](int b) { return __ldcg(p.kv_len + b); }), ++piece) {
    const int end = kv_end(w.len, p.n_new, p.S_max);
    const int safe = keys_all_see(p, w.len);
    const int g = w.u / p.row_groups;
    const int t0 = (w.u - g * p.row_groups) * p.group_pos;
    const bool warp_live = t0 + quarter * 8 < p.T;
    const uint32_t t_o = t_row + 128 * (kS + piece % kO) + 64 * half;  // this half's columns of O
    float m_used = -INFINITY, l_sum = 0.f;
    uint32_t sv[64];
    bool loading = false;  // the tile's S is on its way
    auto load_s = [&](int slot) {
      tc_fence_after();
      const uint32_t at = t_row + slot * 128 + 64 * half;
      tmem_ld32(at, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
      tmem_ld32(at + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
    };
    for (int j = 0; j < w.n; ++j, ++it) {
      const int slot = it % kS;
      const uint32_t t_s = t_row + slot * 128;
      const int key0 = (w.first + j) * kKvTile + 64 * half;
      const bool masked = key0 + 64 > safe;
      KeyWords<2> seen;
      if (masked && warp_live) {
        const int t = t0 + (r >> 2);
        const bool live = t < p.T;
        seen.load(p.mask ? p.mask + (static_cast<size_t>(w.b) * p.T + (live ? t : 0)) * W : nullptr, W, key0 - safe, live);
      }
      if (!loading) ok = wait(bar.s_full(slot), (it / kS) & 1);
      if (!warp_live) {  // rows past the last position: whatever their P is, their O is not used
        if (!ok) break;
        if (lane == 0) arrive_p(slot);
        continue;
      }
      if (!loading) load_s(slot);
      tmem_ld_wait();
      if (masked) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t bits = seen.bits(c, end < 0 ? 0 : p.n_new);
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
      const bool over = j == 0 || m_half > m_used + 8.0f;
      tc_fence_before();
      if (!named_bar_and(bar_id, 64, ok && !over)) {
        if (!(ok = named_bar_and(bar_id, 64, ok))) break;
        *mine = m_half;
        named_bar_sync(bar_id, 64);
        const float m_new = fmaxf(m_used, fmaxf(m_half, *other));
        const float alpha = m_new == -INFINITY ? 0.f : fast_exp2(m_used - m_new);
        m_used = m_new;
        l_sum *= alpha;
        if (j > 0) {
          // O holds the sum through the tile before once its PV, issued behind this tile's S, is done and
          // has released its V (a wait given up shows at the next tile)
          wait(bar.v_empty((it - 1) % kVStages), ((it - 1) / kVStages) & 1);
          tc_fence_after();
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
      const float mu = (m_used == -INFINITY) ? 0.f : m_used;
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
      // the next tile's S, if it is there, comes in under the rest of this one
      const int s_next = (it + 1) % kS;
      loading = j + 1 < w.n &&
                __all_sync(0xffffffffu, mbar_test_wait(bar.s_full(s_next), ((it + 1) / kS) & 1));
      if (loading) load_s(s_next);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_p(slot);
      const float2 l2 = fadd2(fadd2(l4[0], l4[1]), fadd2(l4[2], l4[3]));
      l_sum += l2.x + l2.y;
    }
    // ---------------------------------------------------------------- end of a piece
    const int at = piece % kO;
    // one decision of the row group's warps, with or without live rows, whether a wait was given up
    ok = ok && wait(bar.o_full(at), (piece / kO) & 1);
    if (!(ok = named_bar_and(bar_id, 64, ok))) break;
    if (!warp_live) {
      if (lane == 0) mbar_arrive(bar.o_empty(at));
      continue;
    }
    tc_fence_after();
    uint32_t v[64];
    tmem_ld32(t_o, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
    tmem_ld32(t_o + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
    *mine = l_sum;
    tmem_ld_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar.o_empty(at));
    named_bar_sync(bar_id, 64);
    const float l_other = *other;
    const float l = half ? l_other + l_sum : l_sum + l_other;
    named_bar_sync(bar_id, 64);  // read before the next exchange
    store_piece(p, w, end, g, t0, 0, blockIdx.x, half, quarter, m_used, l, v);
  }
}

__global__ void __launch_bounds__(384, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const CacheAttnParams p) {
  using L = CacheAttnSmem;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const CacheBars bar(smem + L::kBar);
  const CacheRanges ranges(smem + L::kRanges);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) bar.init(4, 8);
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
  ranges.find<1>(p, blockIdx.x, gridDim.x);
  tc_fence_after();
  const uint32_t tmem_base = *bar.tmem_holder();
  // test hook: the last worker loads nothing, its consumers wait out and abort
  const bool no_loads = p.fault && static_cast<int>(blockIdx.x) == ranges.workers() - 1;

  if (warp == 0) {
    if (lane == 0 && !no_loads) produce_k<1>(p, ranges, bar, &tmK, smem + L::kK);
  } else if (warp == 3) {
    if (lane == 0 && !no_loads) produce_vq<kOneTile>(p, ranges, bar, &tmQ, &tmV, smem, 128, kKvHalfBytes, smem + L::kV);
  } else if (warp == 2) {
    clear_v<1>(p, ranges, bar, smem + L::kV);
  } else if (warp == 1) {
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, 0, 0);   // Q, K both K-major
    constexpr uint32_t idesc_pv = idesc_bf16_f32(128, 128, 0, 1);  // P (TMEM), V MN-major
    const uint32_t q_addr = smem_u32(smem), k_addr = smem_u32(smem + L::kK), v_addr = smem_u32(smem + L::kV);
    issue_all<kOneTile, 2>(
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
  } else {
    softmax_halves(p, ranges, bar, tmem_base, reinterpret_cast<float*>(smem + L::kExchange));
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

}  // namespace gqa
