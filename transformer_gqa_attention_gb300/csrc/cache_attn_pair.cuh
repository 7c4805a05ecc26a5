// cache_attn_pair.cuh — attention of 33 and more positions per sequence over caches whose lengths
// differ from sequence to sequence, by CTA pairs (cta_group::2).
//
// A pair is one worker (kv_sched.h) and its units are 64 positions x 4 heads = 256 rows, of which
// CTA r has the 128 of positions 32 r .. 32 r + 31.  The pair's UMMAs read both CTAs' shared memory,
// so each CTA stages half of every key tile (keys 64 r .. + 63 of K, d 64 r .. + 63 of V): a key tile
// costs one SM 32 KB instead of 64.
// A tile's chain is long (K lands, S, softmax, P's word to CTA 0, PV, V's stage and S's buffer free
// again), so its steps are kept apart: S has three buffers and a warp of its own issues it, up to
// three tiles ahead of PV; the softmax's two warpgroups have a tile each on their hands.
// Warps of a CTA (384 threads):
//   warp 0      TMA producer of K and V
//   warp 1      TMEM owner; a unit's queries; in CTA 0 issues the pair's S (M = 256)
//   warp 2      the rows of its half of V that no row sees, in the tiles that have such rows
//   warp 3      in CTA 0 issues the pair's PV
//   warps 4..11 softmax (softmax_in_turn)
// Barriers that the issuers wait on are CTA 0's, and their commits arrive on both CTAs' barriers.
//
// A key tile is 4 x 256 x 128 x 128 FLOP, 1040 cycles of UMMAs, and takes 0.73 us to read; it takes
// 0.75 to 0.8.  32 sequences of 8128 keys and 64 tokens (1.1 GB, 275 GFLOP): 218 us, 5.1 TB/s, where such calls
// follow one another (227 after seconds of them: 1360 W at 1.55 GHz), 190 to 198 in runs of 2.5 ms;
// 32 of 4000 keys 108; one of 32000 keys and 60 tokens 35; 18 of up to 2105 and 103 tokens 58, where a
// unit's begin and end (tail of the last PV, O, stores, the first softmax) cost as much as its tiles.
// Measured against: two row tiles in one CTA (no room for a second S buffer, a ring of two and a half
// tiles) 2.0 us per tile; one issuing warp for S and PV, two buffers of S and two softmax threads per row
// in step with each other 212, 122, 40 and 80 us for the same cases, with the issuers and buffers of
// today 208, 117 and 38.  Rings of 3, 4 and 6 stages: 5, 1 and 3 % slower than 5 for the first.
//
// TMEM columns (each CTA, its own rows): S_0/P_0, S_1/P_1, S_2/P_2 at 0, 128, 256, O at 384.
#pragma once

#include "cache_attn.cuh"
#include "cache_roles.cuh"

namespace gqa {

struct CachePairBars {
  static constexpr int kStages = 5;     // each of K and V
  static constexpr int kS = 3;          // buffers of S
  static constexpr int kRing = 6 + 2 * kS;
  static constexpr int kCount = kRing + 5 * kStages;
  static constexpr int kBytes = 384;
  uint64_t* bars;
  __device__ __forceinline__ explicit CachePairBars(uint8_t* at) : bars(reinterpret_cast<uint64_t*>(at)) {}
  // CTA 0's: both CTAs' bytes of the queries, of K and of V (or, if rows of V are cleared, both CTAs' word
  // that they are)
  __device__ __forceinline__ uint64_t* q_full() const { return bars; }
  __device__ __forceinline__ uint64_t* k_full(int i) const { return bars + kRing + i; }
  __device__ __forceinline__ uint64_t* v_ready(int i) const { return bars + kRing + kStages + i; }
  // CTA 0's: an arrival of every softmax warp of both CTAs that has written its part of P, or read O
  __device__ __forceinline__ uint64_t* p_full(int i) const { return bars + 6 + i; }
  __device__ __forceinline__ uint64_t* o_empty() const { return bars + 1; }
  // each CTA's own
  __device__ __forceinline__ uint64_t* q_empty() const { return bars + 2; }
  __device__ __forceinline__ uint64_t* o_full() const { return bars + 3; }
  __device__ __forceinline__ uint64_t* drain(int i) const { return bars + 4 + i; }
  __device__ __forceinline__ uint64_t* s_full(int i) const { return bars + 6 + kS + i; }
  __device__ __forceinline__ uint64_t* k_empty(int i) const { return bars + kRing + 2 * kStages + i; }
  __device__ __forceinline__ uint64_t* v_empty(int i) const { return bars + kRing + 3 * kStages + i; }
  // the bytes of a half of V of which rows are to be cleared
  __device__ __forceinline__ uint64_t* v_full(int i) const { return bars + kRing + 4 * kStages + i; }
  __device__ __forceinline__ uint32_t* tmem_holder() const { return reinterpret_cast<uint32_t*>(bars + kCount); }
  __device__ __forceinline__ volatile int* abort_flag() const { return reinterpret_cast<volatile int*>(tmem_holder() + 1); }
  __device__ __forceinline__ void init() const {
    for (int i = 0; i < kCount; ++i) {
      const bool p = i >= 6 && i < 6 + kS, v_ready = i >= kRing + kStages && i < kRing + 2 * kStages;
      mbar_init(&bars[i], p ? 8u : i == 1 ? 16u : v_ready ? 2u : 1u);
    }
    *abort_flag() = 0;
    fence_mbar_init();
  }
};

// A place in a ring of N and the parity of its phase.
template <int N>
struct RingPlace {
  int i = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++i == N) {
      i = 0;
      parity ^= 1u;
    }
  }
};

struct CachePairSmem {
  static constexpr int kStage = kKvTileBytes / 2;  // half a key tile of K or V
  static constexpr int kK = kKvTileBytes;          // behind the query tile
  static constexpr int kV = kK + CachePairBars::kStages * kStage;
  static constexpr int kBar = kV + CachePairBars::kStages * kStage;
  static constexpr int kRanges = kBar + CachePairBars::kBytes;
  static constexpr int kExchange = kRanges + CacheRanges::kBytes;  // [2 halves][128 rows] floats
  static constexpr int kBytes = kExchange + 2 * 128 * 4 + 1024;
};

// The softmax warps of CTA `rank` (warps 4..11): rows are positions t0 .. t0 + 31 of a unit, one thread
// per row.  Warps 4..7 and 8..11 take the worker's tiles in turn, so that one set's loads, maxima and
// waits pass under the other's exponentials.  Both write P for one O and so with one running maximum m,
// which a set hands on to the other with its tile's decision, before its exponentials; each sums its own
// tiles' l.  m is only needed to keep 2^(c s - m) in range: it follows the scores when a row's tile has
// one that passes m + 8, and the set that finds it rescales O.
// A wait given up ends the walk at the end of the piece: until then the sets go on handing m to each
// other, as barriers between them have no time limit.
template <typename FP, typename FO>
__device__ __forceinline__ void softmax_in_turn(const CacheAttnParams& p, const CacheRanges& ranges,
                                                const CachePairBars& bar, uint32_t tmem_base, float* exchange, int rank,
                                                int worker, FP arrive_p, FO arrive_o) {
  constexpr int kS = CachePairBars::kS, kStages = CachePairBars::kStages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int set = (warp - 4) >> 2;    // also: which 64 columns of O at the end of a piece
  const int quarter = warp & 3;
  const int r = quarter * 32 + lane;  // row of the tile: position r / 4, head r & 3
  const int bar_id = 1 + quarter;     // the two warps that share rows
  const int give = 5 + 4 * set + quarter, take = 5 + 4 * (set ^ 1) + quarter;  // m from set to set
  const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
  const uint32_t t_o = t_row + kS * 128;
  float* mine = exchange + set * 128 + r;
  volatile const float* other = exchange + (set ^ 1) * 128 + r;
  const int W = (p.T + 31) / 32;
  const int units = p.n_kv * p.row_groups;
  volatile int* abort_flag = bar.abort_flag();
  auto wait = [&](uint64_t* b, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(b, parity, abort_flag, p.status));
  };
  KvWalk w = ranges.walk(0, p);
  int it = 0, piece = 0;
  for (; !w.done(); w.next(units, p.n_new, p.S_max, [&](int b) { return __ldcg(p.kv_len + b); }), ++piece) {
    const int end = kv_end(w.len, p.n_new, p.S_max);
    const int safe = keys_all_see(p, w.len);
    const int g = w.u / p.row_groups;
    const int t0 = (w.u - g * p.row_groups) * p.group_pos + 32 * rank;
    const int t = t0 + (r >> 2);
    const bool warp_live = t0 + quarter * 8 < p.T, live = t < p.T;
    float m_used = -INFINITY, l_sum = 0.f;
    bool ok = true;
    for (int j = (it & 1) ^ set; j < w.n; j += 2) {
      const int tile = it + j, slot = tile % kS;
      const uint32_t t_s = t_row + 128 * slot;
      const int key0 = (w.first + j) * kKvTile;
      const bool masked = key0 + kKvTile > safe;
      KeyWords<4> seen;
      if (masked && warp_live)
        seen.load(p.mask ? p.mask + (static_cast<size_t>(w.b) * p.T + (live ? t : 0)) * W : nullptr, W, key0 - safe, live);
      ok = ok && wait(bar.s_full(slot), (tile / kS) & 1);
      if (!warp_live) {  // rows past the last position: whatever their P is, their O is not used
        if (!ok) break;
        if (lane == 0) arrive_p(slot);
        continue;
      }
      if (!ok) {
        if (j > 0) named_bar_sync(take, 64);
        if (j + 1 < w.n) named_bar_arrive(give, 64);
        continue;
      }
      tc_fence_after();
      uint32_t sv[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(t_s + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&sv[32 * c]));
      tmem_ld_wait();
      if (masked) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
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
      for (int k = 0; k < 60; ++k)
        m8[k & 7] = max3f(m8[k & 7], __uint_as_float(sv[8 + 2 * k]), __uint_as_float(sv[9 + 2 * k]));
      const float mx = max3f(max3f(m8[0], m8[1], m8[2]), max3f(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
      const float m_tile = mx * p.scale_log2;
      float m_prev = m_tile;
      if (j > 0) {
        named_bar_sync(take, 64);
        m_prev = *other;
      }
      const bool grow = m_tile > m_prev + 8.0f;
      const float m = grow ? m_tile : m_prev;
      if (j + 1 < w.n) {
        *mine = m;
        named_bar_arrive(give, 64);
      }
      l_sum = m == -INFINITY ? 0.f : l_sum * fast_exp2(m_used - m);
      m_used = m;
      if (__any_sync(0xffffffffu, grow)) {
        // O holds the sum through the tile before, of the other set, once its PV is done and has released
        // its V (a wait given up shows at the next tile)
        wait(bar.v_empty((tile - 1) % kStages), ((tile - 1) / kStages) & 1);
        tc_fence_after();
        const float alpha = grow ? fast_exp2(m_prev - m) : 1.f;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          tmem_ld32(t_o + c * 32, v);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha);
          tmem_st32(t_o + c * 32, v);
        }
      }
      const float mu = (m == -INFINITY) ? 0.f : m;
      const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
      const float2 nmu2 = make_float2(-mu, -mu);
      float2 l4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
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
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_p(slot);
      const float2 l2 = fadd2(fadd2(l4[0], l4[1]), fadd2(l4[2], l4[3]));
      l_sum += l2.x + l2.y;
    }
    it += w.n;
    // ---------------------------------------------------------------- end of a piece
    // one decision of the two warps, with or without live rows, whether a wait was given up
    ok = ok && wait(bar.o_full(), piece & 1);
    if (!named_bar_and(bar_id, 64, ok)) break;
    if (!warp_live) {
      if (lane == 0) arrive_o();
      continue;
    }
    tc_fence_after();
    uint32_t v[64];
    tmem_ld32(t_o + 64 * set, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
    tmem_ld32(t_o + 64 * set + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
    *mine = m_used;  // -inf if the set had no tile
    tmem_ld_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) arrive_o();
    named_bar_sync(bar_id, 64);
    const float m = fmaxf(m_used, *other);  // the last tile's
    named_bar_sync(bar_id, 64);
    const float l_mine = m == -INFINITY ? 0.f : l_sum * fast_exp2(m_used - m);
    *mine = l_mine;
    named_bar_sync(bar_id, 64);
    const float l_other = *other;
    const float l = set ? l_other + l_mine : l_mine + l_other;
    named_bar_sync(bar_id, 64);  // read before the next exchange
    store_piece(p, w, end, g, t0, rank, worker, set, quarter, m, l, v);
  }
}

// tmK: boxes of 64 keys; tmV: of 128
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(384, 1)
    cache_attn_pair_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const CacheAttnParams p) {
  using L = CachePairSmem;
  constexpr int kStages = CachePairBars::kStages, kS = CachePairBars::kS;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const CachePairBars bar(smem + L::kBar);
  const CacheRanges ranges(smem + L::kRanges);
  volatile int* abort_flag = bar.abort_flag();
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int worker = blockIdx.x >> 1;

  if (threadIdx.x == 0) bar.init();
  if (warp == 1) {
    tmem_alloc_pair(bar.tmem_holder(), 512);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  griddep_launch_dependents();
  griddep_wait();  // lengths, queries and the new cache entries; the scratch of the call before
  tc_fence_before();
  ranges.find<1>(p, worker, gridDim.x >> 1);
  cluster_sync();  // the peer's barriers are initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = *bar.tmem_holder();
  const uint64_t policy = kv_policy(p);
  // test hook: the last pair loads nothing, its consumers wait out and abort
  const bool no_loads = p.fault && worker == ranges.workers() - 1;
  auto cta0 = [&](uint64_t* b) { return mapa_shared(smem_u32(b), 0); };
  // a whole warp's waits
  auto wait = [&](uint64_t* b, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(b, parity, abort_flag, p.status));
  };
  auto wait_cluster = [&](uint64_t* b, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_cluster(b, parity, abort_flag, p.status));
  };
  // a warp that issued UMMAs, after a wait that was given up: they finish before TMEM is released
  auto drain = [&](uint64_t* b) {
    if (!__any_sync(0xffffffffu, *abort_flag != 0)) return;
    if (elect_one_sync()) umma_commit_pair(b, 0x1);
    __syncwarp();
    mbar_wait_drain(b, 0);
  };

  const int units = p.n_kv * p.row_groups;
  auto next = [&](KvWalk& w) {
    w.next(units, p.n_new, p.S_max, [&](int b) { return __ldcg(p.kv_len + b); });
  };
  // tile t of a piece has rows of V that no row of the product sees
  auto cleared = [&](const KvWalk& w, int t) { return (t + 1) * kKvTile > keys_all_see(p, w.len); };

  // registers: 168 x 384 at launch >= 72 x 128 (warps 0..3) + 208 x 256 (the softmax warps)
  if (warp < 4) {
    setmaxnreg_dec<72>();
    if (warp == 0) {
      if (lane == 0 && !no_loads) {
        // ---------------------------------------------------------------- K and V producer
        // K runs a tile ahead of V (one to four: within 2 %).
        constexpr int kAhead = 1;
        KvWalk kw = ranges.walk(0, p), vw = kw;
        RingPlace<kStages> k, v;
        int kj = 0, k_asked = 0, v_asked = 0;
        uint32_t v_own = 0, own_parity = 0;  // of V's places: rows are cleared; parity of v_full's last phase
        auto ask_k = [&] {
          if (kw.done()) return true;
          if (!mbar_wait(bar.k_empty(k.i), k.parity ^ 1u, abort_flag, p.status)) return false;
          if (rank == 0) mbar_arrive_expect_tx(bar.k_full(k.i), 2 * L::kStage);
          uint8_t* dst = smem + L::kK + k.i * L::kStage;
          const int g = kw.u / p.row_groups, key0 = (kw.first + kj) * kKvTile + 64 * rank;
          tma_load_4d_pair_hint(dst, &tmK, cta0(bar.k_full(k.i)), 0, g, key0, kw.b, policy);
          tma_load_4d_pair_hint(dst + L::kStage / 2, &tmK, cta0(bar.k_full(k.i)), 64, g, key0, kw.b, policy);
          ++k_asked;
          k.next();
          if (++kj == kw.n) {
            kj = 0;
            next(kw);
          }
          return true;
        };
        bool ok = true;
        for (int i = 0; i < kAhead && ok; ++i) ok = ask_k();
        for (; ok && !vw.done(); next(vw)) {
          for (int j = 0; j < vw.n; ++j) {
            if (!(ok = ask_k() && mbar_wait(bar.v_empty(v.i), v.parity ^ 1u, abort_flag, p.status))) break;
            uint8_t* dst = smem + L::kV + v.i * L::kStage;
            const int g = vw.u / p.row_groups, key0 = (vw.first + j) * kKvTile;
            if (cleared(vw, vw.first + j)) {
              v_own |= 1u << v.i;
              own_parity ^= 1u << v.i;
              mbar_arrive_expect_tx(bar.v_full(v.i), L::kStage);
              tma_load_4d_hint(dst, &tmV, bar.v_full(v.i), 64 * rank, g, key0, vw.b, policy);
            } else {
              v_own &= ~(1u << v.i);
              if (rank == 0) {
                mbar_arrive_expect_tx(bar.v_ready(v.i), 2 * L::kStage);
                mbar_arrive(bar.v_ready(v.i));
              }
              tma_load_4d_pair_hint(dst, &tmV, cta0(bar.v_ready(v.i)), 64 * rank, g, key0, vw.b, policy);
            }
            ++v_asked;
            v.next();
          }
          if (!ok) break;
        }
        // let copies still in flight land before the pair leaves (CTA 0's barriers count both CTAs' bytes)
        if (*abort_flag) {
          for (int i = max(0, k_asked - kStages); rank == 0 && i < k_asked; ++i)
            mbar_wait_drain(bar.k_full(i % kStages), (i / kStages) & 1);
          for (int i = max(0, v_asked - kStages); i < v_asked; ++i) {
            const int at = i % kStages;
            if ((v_own >> at) & 1)
              mbar_wait_drain(bar.v_full(at), ((own_parity >> at) & 1) ^ 1u);
            else if (rank == 0)
              mbar_wait_drain(bar.v_ready(at), (i / kStages) & 1);
          }
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------------ queries; S = Q K^T of the pair
      // The whole warp runs the loop (its waits are warp-uniform); one elected lane issues.  S is up to
      // three tiles ahead of PV, so that a unit's queries arrive under the softmax of the unit before.
      constexpr uint32_t idesc_s = idesc_bf16_f32(256, 128, 0, 0);  // Q, K both K-major
      const uint64_t q_desc = sdesc_sw128(smem_u32(smem), 0, 1024);
      const uint32_t k_addr = smem_u32(smem + L::kK);
      RingPlace<kStages> k, v;  // v: of the PV whose P the tile's S takes the place of
      RingPlace<kS> s;
      KvWalk w = ranges.walk(0, p);
      int piece = 0, free_s = kS;
      bool ok = !no_loads;
      for (; ok && !w.done(); next(w), ++piece) {
        if (piece > 0 && !(ok = wait(bar.q_empty(), (piece - 1) & 1))) break;
        if (elect_one_sync()) {
          const int g = w.u / p.row_groups, t0 = (w.u - g * p.row_groups) * 64 + 32 * rank;
          if (rank == 0) mbar_arrive_expect_tx(bar.q_full(), 2 * kKvTileBytes);
          tma_load_4d_pair(smem, &tmQ, cta0(bar.q_full()), 0, 4 * g, t0, w.b);
          tma_load_4d_pair(smem + kKvHalfBytes, &tmQ, cta0(bar.q_full()), 64, 4 * g, t0, w.b);
        }
        __syncwarp();
        if (rank == 1) continue;
        if (!(ok = wait(bar.q_full(), piece & 1))) {
          if (lane == 0) mbar_wait_drain(bar.q_full(), piece & 1);  // (both CTAs' bytes)
          break;
        }
        for (int j = 0; j < w.n; ++j) {
          if (!(ok = wait(bar.k_full(k.i), k.parity))) break;
          if (free_s > 0) {
            --free_s;
          } else {
            if (!(ok = wait(bar.v_empty(v.i), v.parity))) break;
            v.next();
          }
          tc_fence_after();
          if (elect_one_sync()) {
            const uint64_t kd = sdesc_sw128(k_addr + k.i * L::kStage, 0, 1024);
  #pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma_ss_pair(tmem_base + s.i * 128, q_desc + (((kk >> 2) * kKvHalfBytes + (kk & 3) * 32) >> 4),
                           kd + (((kk >> 2) * (L::kStage / 2) + (kk & 3) * 32) >> 4), idesc_s, kk != 0);
            umma_commit_pair(bar.s_full(s.i), 0x3);
            umma_commit_pair(bar.k_empty(k.i), 0x3);
            if (j == w.n - 1) umma_commit_pair(bar.q_empty(), 0x3);
          }
          __syncwarp();
          k.next();
          s.next();
        }
      }
      if (rank == 0) drain(bar.drain(0));
    } else if (warp == 2) {
      // ------------------------------------------------------------------ V rows nobody sees
      ClearRows clear;
      uint32_t own_parity = 0;  // of V's places: parity of v_full's next phase
      int it0 = 0;              // tiles before the piece
      KvWalk w = ranges.walk(0, p);
      if (rank == 0 && lane == 0 && w.done()) p.merge[worker] = make_int4(-1, 0, 0, 0);
      bool ok = true;
      for (; ok && !w.done(); it0 += w.n, next(w)) {
        if (rank == 0 && lane == 0 && w.after == 0) p.merge[worker] = goes_on(ranges, w, worker);
        for (int j = max(0, keys_all_see(p, w.len) / kKvTile - w.first); j < w.n; ++j) {
          const CacheLane l{w, j, 0};
          clear.prepare(p, l);
          const int vs = (it0 + j) % kStages;
          const uint32_t parity = (own_parity >> vs) & 1;
          own_parity ^= 1u << vs;
          if (!(ok = wait(bar.v_full(vs), parity))) break;
          const bool any = clear.rows<8>(p, l, [&](int r, int c) {
            return smem + L::kV + vs * L::kStage + r * 128 + c * 16;  // this CTA's 64 columns
          });
          if (any) {
            fence_proxy_async_smem();
            __syncwarp();
          }
          // this CTA's half of V, as it landed or as cleared here, is read by products that CTA 0 issues: ordered
          // at cluster scope in either case
          if (lane == 0) mbar_arrive_cluster(cta0(bar.v_ready(vs)));
        }
      }
    } else if (warp == 3) {
      if (rank == 0) {
        // ---------------------------------------------------------------- O += P V of the pair
        constexpr uint32_t idesc_pv = idesc_bf16_f32(256, 128, 0, 1);  // P (TMEM), V MN-major
        const uint32_t v_addr = smem_u32(smem + L::kV);
        RingPlace<kStages> v;
        RingPlace<kS> s;
        KvWalk w = ranges.walk(0, p);
        int piece = 0;
        bool ok = true;
        for (; ok && !w.done(); next(w), ++piece) {
          // the piece's O takes the place of the piece's before
          if (piece > 0 && !(ok = wait(bar.o_empty(), (piece - 1) & 1))) break;
          for (int j = 0; j < w.n; ++j) {
            const bool there = cleared(w, w.first + j) ? wait_cluster(bar.v_ready(v.i), v.parity) : wait(bar.v_ready(v.i), v.parity);
            if (!(ok = there && wait(bar.p_full(s.i), s.parity))) break;
            tc_fence_after();
            if (elect_one_sync()) {
              const uint64_t vd = sdesc_sw128(v_addr + v.i * L::kStage, L::kStage, 1024);
  #pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                umma_ts_pair(tmem_base + kS * 128, tmem_base + s.i * 128 + kk * 8, vd + ((kk * 2048) >> 4), idesc_pv,
                             j + kk != 0);
              umma_commit_pair(bar.v_empty(v.i), 0x3);
              if (j == w.n - 1) umma_commit_pair(bar.o_full(), 0x3);
            }
            __syncwarp();
            v.next();
            s.next();
          }
        }
        drain(bar.drain(1));
      }
    }
  } else {
    setmaxnreg_inc<208>();
    softmax_in_turn(
        p, ranges, bar, tmem_base, reinterpret_cast<float*>(smem + L::kExchange), rank, worker,
        [&](int slot) { mbar_arrive_remote(cta0(bar.p_full(slot))); },
        [&] { mbar_arrive_remote(cta0(bar.o_empty())); });
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the pair's UMMAs or remote arrivals are live
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

}  // namespace gqa
