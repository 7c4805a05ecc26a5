// cache_attn_pair.cuh — attention of 33 and more positions per sequence over caches whose lengths
// differ from sequence to sequence, by CTA pairs (cta_group::2).
//
// A pair is one worker (kv_sched.h) and its units are 64 positions x 4 heads = 256 rows, of which
// CTA r has the 128 of positions 32 r .. 32 r + 31.  The pair's UMMAs read both CTAs' shared memory,
// so each CTA stages half of every key tile (keys 64 r .. + 63 of K, d 64 r .. + 63 of V) and a key
// tile costs one SM 32 KB instead of 64: ten 16 KB stages are 160 KB in flight, and the softmax of a
// CTA has one row tile per key tile, whose S alternates between two buffers.  With two row tiles in
// one CTA and the same shared memory the ring held two and a half key tiles, and S could not be
// buffered: 2.0 us per key tile and SM, against 1.47 us to read it.
// Roles per CTA as in cache_roles.cuh, but
//   warp 1      of CTA 0 issues the pair's UMMAs (M = 256), of CTA 1 only keeps its TMEM
//   warp 2      waits for every V half, clears rows if need be, and tells CTA 0
// Barriers that the issuer waits on are CTA 0's, and its commits arrive on both CTAs' barriers.
//
// TMEM columns (each CTA, its own rows): S_0/P_0 at 0, S_1/P_1 at 128, O_0 at 256, O_1 at 384.
#pragma once

#include "cache_attn.cuh"
#include "cache_roles.cuh"

namespace gqa {

struct CachePairBars {
  static constexpr int kStages = 5;  // each of K and V
  static constexpr int kV = kStages;
  static constexpr int kCount = 15 + 5 * kStages;
  static constexpr int kBytes = 384;
  uint64_t* bars;
  __device__ __forceinline__ explicit CachePairBars(uint8_t* at) : bars(reinterpret_cast<uint64_t*>(at)) {}
  // CTA 0's: both CTAs' bytes of the queries and of K, and both CTAs' word that V is there and clear
  __device__ __forceinline__ uint64_t* q_full(int i) const { return bars + i; }
  __device__ __forceinline__ uint64_t* k_full(int i) const { return bars + 15 + i; }
  __device__ __forceinline__ uint64_t* v_ready(int i) const { return bars + 15 + kStages + i; }
  // CTA 0's: an arrival of every softmax warp of both CTAs that writes P's half, or reads O
  __device__ __forceinline__ uint64_t* p_lo(int i) const { return bars + 2 + i; }
  __device__ __forceinline__ uint64_t* p_hi(int i) const { return bars + 4 + i; }
  __device__ __forceinline__ uint64_t* o_empty(int i) const { return bars + 6 + i; }
  // each CTA's own
  __device__ __forceinline__ uint64_t* q_empty(int i) const { return bars + 8 + i; }
  __device__ __forceinline__ uint64_t* s_full(int i) const { return bars + 10 + i; }
  __device__ __forceinline__ uint64_t* o_full(int i) const { return bars + 12 + i; }
  __device__ __forceinline__ uint64_t* drain() const { return bars + 14; }
  __device__ __forceinline__ uint64_t* k_empty(int i) const { return bars + 15 + 2 * kStages + i; }
  __device__ __forceinline__ uint64_t* v_full(int i) const { return bars + 15 + 3 * kStages + i; }
  __device__ __forceinline__ uint64_t* v_empty(int i) const { return bars + 15 + 4 * kStages + i; }
  __device__ __forceinline__ uint32_t* tmem_holder() const { return reinterpret_cast<uint32_t*>(bars + kCount); }
  __device__ __forceinline__ volatile int* abort_flag() const { return reinterpret_cast<volatile int*>(tmem_holder() + 1); }
  __device__ __forceinline__ void init() const {
    for (int i = 0; i < kCount; ++i) {
      const bool p_half = i >= 2 && i < 6, o = i == 6 || i == 7;
      const bool v_ready = i >= 15 + kStages && i < 15 + 2 * kStages;
      mbar_init(&bars[i], p_half ? 8u : o ? 16u : v_ready ? 2u : 1u);
    }
    *abort_flag() = 0;
    fence_mbar_init();
  }
};

struct CachePairSmem {
  static constexpr int kStage = kKvTileBytes / 2;  // half a key tile of K or V
  static constexpr int kK = 2 * kKvTileBytes;      // behind two query tiles
  static constexpr int kV = kK + CachePairBars::kStages * kStage;
  static constexpr int kBar = kV + CachePairBars::kStages * kStage;
  static constexpr int kRanges = kBar + CachePairBars::kBytes;
  static constexpr int kExchange = kRanges + CacheRanges::kBytes;  // [2 halves][128 rows] floats
  static constexpr int kBytes = kExchange + 2 * 128 * 4 + 1024;
};

// tmK: boxes of 64 keys; tmV: of 128
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(384, 1)
    cache_attn_pair_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const CacheAttnParams p) {
  using L = CachePairSmem;
  constexpr int kStages = CachePairBars::kStages;
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

  if (warp == 0) {
    if (lane == 0 && !no_loads) {
      // ---------------------------------------------------------------- K producer
      CacheTiles<1> tiles(p, ranges);
      int it = 0;
      tiles.each([&](auto, CacheLane& l) {
        const int st = it % kStages;
        if (!mbar_wait(bar.k_empty(st), ((it / kStages) & 1) ^ 1u, abort_flag, p.status)) return false;
        if (rank == 0) mbar_arrive_expect_tx(bar.k_full(st), 2 * L::kStage);
        uint8_t* dst = smem + L::kK + st * L::kStage;
        const int g = l.w.u / p.row_groups, key0 = (l.w.first + l.j) * kKvTile + 64 * rank;
        tma_load_4d_pair_hint(dst, &tmK, cta0(bar.k_full(st)), 0, g, key0, l.w.b, policy);
        tma_load_4d_pair_hint(dst + L::kStage / 2, &tmK, cta0(bar.k_full(st)), 64, g, key0, l.w.b, policy);
        ++it;
        return true;
      });
      // let copies still in flight land before the pair leaves (CTA 0's barriers count both CTAs' bytes)
      if (*abort_flag && rank == 0)
        for (int i = max(0, it - kStages); i < it; ++i) mbar_wait_drain(bar.k_full(i % kStages), (i / kStages) & 1);
    }
  } else if (warp == 3) {
    if (lane == 0 && !no_loads) {
      // ---------------------------------------------------------------- V and query producer
      CacheTiles<1> tiles(p, ranges);
      int it = 0, asked = 0;
      tiles.each([&](auto, CacheLane& l) {
        const int g = l.w.u / p.row_groups;
        if (l.j == 0) {
          const int t0 = (l.w.u - g * p.row_groups) * 64 + 32 * rank;
          const int at = l.piece & 1, turn = l.piece >> 1;
          if (turn > 0 && !mbar_wait(bar.q_empty(at), (turn - 1) & 1, abort_flag, p.status)) return false;
          if (rank == 0) mbar_arrive_expect_tx(bar.q_full(at), 2 * kKvTileBytes);
          uint8_t* dst = smem + at * kKvTileBytes;
          tma_load_4d_pair(dst, &tmQ, cta0(bar.q_full(at)), 0, 4 * g, t0, l.w.b);
          tma_load_4d_pair(dst + kKvHalfBytes, &tmQ, cta0(bar.q_full(at)), 64, 4 * g, t0, l.w.b);
          ++asked;
        }
        const int st = it % kStages;
        if (!mbar_wait(bar.v_empty(st), ((it / kStages) & 1) ^ 1u, abort_flag, p.status)) return false;
        mbar_arrive_expect_tx(bar.v_full(st), L::kStage);
        tma_load_4d_hint(smem + L::kV + st * L::kStage, &tmV, bar.v_full(st), 64 * rank, g,
                         (l.w.first + l.j) * kKvTile, l.w.b, policy);
        ++it;
        return true;
      });
      if (*abort_flag) {
        for (int i = max(0, it - kStages); i < it; ++i) mbar_wait_drain(bar.v_full(i % kStages), (i / kStages) & 1);
        if (rank == 0)
          for (int i = max(0, asked - 2); i < asked; ++i) mbar_wait_drain(bar.q_full(i & 1), (i >> 1) & 1);
      }
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------------ V rows nobody sees
    CacheTiles<1> tiles(p, ranges);
    ClearRows clear;
    int it = 0;
    if (rank == 0 && lane == 0 && tiles.l0.w.done()) p.merge[worker] = make_int4(-1, 0, 0, 0);
    tiles.each([&](auto, CacheLane& l) {
      if (rank == 0 && lane == 0 && l.j == 0 && l.w.after == 0) p.merge[worker] = goes_on(ranges, l.w, worker);
      const bool fix = clear.prepare(p, l);
      const int st = it % kStages;
      if (!__all_sync(0xffffffffu, mbar_wait(bar.v_full(st), (it / kStages) & 1, abort_flag, p.status))) return false;
      if (fix) clear.rows(p, l, [&](int r, int c) -> uint8_t* {
        return c < 8 ? smem + L::kV + st * L::kStage + r * 128 + c * 16 : nullptr;  // this CTA's 64 columns
      });
      // rows cleared here are read by the pair's UMMAs: ordered at cluster scope
      if (fix) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(cta0(bar.v_ready(st)));
      } else {
        if (lane == 0) mbar_arrive_remote(cta0(bar.v_ready(st)));
      }
      ++it;
      return true;
    });
  } else if (warp == 1) {
    if (rank == 0) {
      // ------------------------------------------------------------------ UMMA issuer of the pair
      // The whole warp runs the loop (its waits are warp-uniform); one elected lane issues.
      constexpr uint32_t idesc_s = idesc_bf16_f32(256, 128, 0, 0);   // Q, K both K-major
      constexpr uint32_t idesc_pv = idesc_bf16_f32(256, 128, 0, 1);  // P (TMEM), V MN-major
      const uint32_t q_addr = smem_u32(smem), k_addr = smem_u32(smem + L::kK), v_addr = smem_u32(smem + L::kV);
      CacheTiles<1> tiles(p, ranges);
      auto wait = [&](uint64_t* b, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(b, parity, abort_flag, p.status));
      };
      auto wait_cluster = [&](uint64_t* b, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait_cluster(b, parity, abort_flag, p.status));
      };
      struct Pending {
        int it, piece;
        bool first, last, fix;  // first / last tile of the piece; rows of V are cleared
      } pend{};
      bool has_pend = false;
      auto issue_pv = [&] {
        const Pending d = pend;
        has_pend = false;
        const int slot = d.it & 1, o = d.piece & 1, vs = d.it % kStages;
        // a new O takes the place of the one two pieces before
        if (d.first && d.piece > 1 && !wait(bar.o_empty(o), ((d.piece >> 1) - 1) & 1)) return false;
        if (!(d.fix ? wait_cluster(bar.v_ready(vs), (d.it / kStages) & 1) : wait(bar.v_ready(vs), (d.it / kStages) & 1)))
          return false;
        const uint64_t vd = sdesc_sw128(v_addr + vs * L::kStage, L::kStage, 1024);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          if (!wait(hf ? bar.p_hi(slot) : bar.p_lo(slot), (d.it >> 1) & 1)) return false;
          tc_fence_after();
          if (elect_one_sync()) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int kk = 4 * hf + i;
              umma_ts_pair(tmem_base + 256 + o * 128, tmem_base + slot * 128 + kk * 8, vd + ((kk * 2048) >> 4), idesc_pv,
                           !(d.first && kk == 0));
            }
            if (hf) {
              umma_commit_pair(bar.v_empty(vs), 0x3);
              if (d.last) umma_commit_pair(bar.o_full(o), 0x3);
            }
          }
          __syncwarp();
        }
        return true;
      };
      int it = 0;
      const bool ok = tiles.each([&](auto, CacheLane& l) {
        const bool first = l.j == 0, last = l.j == l.w.n - 1;
        const int ks = it % kStages, slot = it & 1, at = l.piece & 1;
        if (first && !wait(bar.q_full(at), (l.piece >> 1) & 1)) return false;
        if (!wait(bar.k_full(ks), (it / kStages) & 1)) return false;
        tc_fence_after();
        if (elect_one_sync()) {
          const uint64_t qd = sdesc_sw128(q_addr + at * kKvTileBytes, 0, 1024);
          const uint64_t kd = sdesc_sw128(k_addr + ks * L::kStage, 0, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_ss_pair(tmem_base + slot * 128, qd + (((kk >> 2) * kKvHalfBytes + (kk & 3) * 32) >> 4),
                         kd + (((kk >> 2) * (L::kStage / 2) + (kk & 3) * 32) >> 4), idesc_s, kk != 0);
          umma_commit_pair(bar.s_full(slot), 0x3);
          umma_commit_pair(bar.k_empty(ks), 0x3);
          if (last) umma_commit_pair(bar.q_empty(at), 0x3);
        }
        __syncwarp();
        if (has_pend && !issue_pv()) return false;
        pend = Pending{it, l.piece, first, last, (l.w.first + l.j + 1) * kKvTile > keys_all_see(p, l.w.len)};
        has_pend = true;
        ++it;
        return true;
      });
      if (ok && has_pend) issue_pv();
      if (__any_sync(0xffffffffu, *abort_flag != 0)) {  // let issued UMMAs finish before TMEM is released
        if (elect_one_sync()) umma_commit_pair(bar.drain(), 0x1);
        __syncwarp();
        mbar_wait_drain(bar.drain(), 0);
      }
    }
  } else {
    softmax_halves(
        p, ranges, bar, tmem_base, reinterpret_cast<float*>(smem + L::kExchange), rank, worker,
        [&](uint64_t* b, uint32_t parity) { return mbar_wait(b, parity, abort_flag, p.status); },
        [&](int slot, int half) { mbar_arrive_remote(cta0(half ? bar.p_hi(slot) : bar.p_lo(slot))); },
        [&](int at) { mbar_arrive_remote(cta0(bar.o_empty(at))); });
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
