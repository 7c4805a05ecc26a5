// cache_attn.cuh — attention of a few positions per sequence over caches whose lengths differ from
// sequence to sequence: a tree of drafted tokens (each row sees the prefix and the drafted tokens
// its mask names), and a decode step that also hands on its scores, from which the key weights are
// accumulated.
//
// The four query heads of a kv head read the same keys and values, so the tensor core's 128 rows
// are 32 positions x 4 heads: row 4t + h.  Every K/V byte then serves all rows of up to 32 (or,
// with two row tiles, 64) positions, and the kernel is bound by reading the cache once while the
// drafts are that small: 4 T rows do 4 T x 128 x 4 FLOP per key of 512 bytes.
//
// Persistent CTAs, one per SM, share the key tiles of all sequences evenly (kv_sched.h).  Roles:
//   warp 0      TMA producer of the 128-key K and V tiles (rings of 2 and 3), running ahead over
//               the ends of units
//   warp 1      TMEM owner and UMMA issuer: S = Q K^T into TMEM, O += P V with P read from TMEM.
//               The next item's S is issued before the last one's PV, so the tensor core works
//               while a softmax runs.
//   warp 2      zeroes the rows of a V tile that no row sees (past the end of the sequence, or
//               drafted positions that nobody's mask names): their weight is 0, but 0 x NaN is not
//   warp 3      TMA of each unit's queries, as soon as the last S of the unit before has read its
//   warps 4..7, 8..11  two softmax slots, one thread per row, as in flash_prefill.cuh
// What the two slots are depends on the rows (kPair):
//   kPair = false (at most 32 positions): the two slots take the unit's key tiles in turn, each
//     with its own running maximum, sum and O; both read both O from TMEM at the end of a piece
//     and merge them, 64 columns each.
//   kPair = true: slot i has positions 32 i .. 32 i + 31 of a group of 64, and both work on the
//     same key tile.
// A piece that is a whole unit is normalised and stored to h; another leaves an unnormalised O
// (fp32) with its maximum and sum in the scratch, which cache_merge_kernel joins.
//
// TMEM columns: S_0/P_0 at 0, S_1/P_1 at 128, O_0 at 256, O_1 at 384.
#pragma once

#include "kv_sched.h"
#include "params.h"
#include "ptx.cuh"

namespace gqa {

template <bool kPair>
struct CacheAttnSmem {
  static constexpr int kTile = 128 * 128 * 2;  // 128 x 128 bf16 (two 64-column halves)
  static constexpr int kHalf = 128 * 64 * 2;
  static constexpr int kQTiles = kPair ? 2 : 1;
  static constexpr int kKStages = 2;
  static constexpr int kVStages = 3;
  static constexpr int kK = kQTiles * kTile;
  static constexpr int kV = kK + kKStages * kTile;
  static constexpr int kBar = kV + kVStages * kTile;
  static constexpr int kSched = kBar + 256;      // 16 ints of the scan, 8 of the range
  static constexpr int kMl = kSched + 128;       // [2 slots][128 rows] (maximum, sum), kPair = false
  static constexpr int kBytes = kMl + (kPair ? 0 : 2 * 128 * 8) + 1024;
};

// Visibility bits of the 32 keys whose drafted index starts at `base` (negative: prefix, always
// seen) for a mask row of W words over n_new drafted positions; a row without a mask (null) that
// is live sees all n_new.
__device__ __forceinline__ uint32_t key_bits(const uint32_t* mask, int W, int n_new, int base, bool live) {
  if (base <= -32) return 0xFFFFFFFFu;
  if (base >= n_new) return 0u;
  const int q = base >> 5;  // floor: -1 where the word straddles the prefix
  const uint32_t none = !live ? 0u : 0xFFFFFFFFu;
  const uint32_t lo = q < 0 ? 0xFFFFFFFFu : (mask ? (live ? __ldcg(mask + q) : 0u) : none);
  const uint32_t hi = q + 1 < W ? (mask ? (live ? __ldcg(mask + q + 1) : 0u) : none) : 0u;
  const uint32_t bits = __funnelshift_r(lo, hi, base & 31);
  const int rem = n_new - base;
  return rem < 32 ? bits & ((1u << rem) - 1u) : bits;
}

template <bool kPair, bool kScores>
__global__ void __launch_bounds__(384, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const CacheAttnParams p) {
  static_assert(!(kPair && kScores), "scores are handed on for one position per sequence");
  using L = CacheAttnSmem<kPair>;
  constexpr int kKS = L::kKStages, kVS = L::kVStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* q_full = bars + 0;
  uint64_t* q_empty = bars + 1;
  uint64_t* k_full = bars + 2;    // [2]
  uint64_t* k_empty = bars + 4;   // [2]
  uint64_t* v_full = bars + 6;    // [3]
  uint64_t* v_empty = bars + 9;   // [3], 2 arrivals: the PV that used the tile, and warp 2
  uint64_t* v_fixed = bars + 12;  // [3]
  uint64_t* s_full = bars + 15;   // [2] slots
  uint64_t* o_full = bars + 17;
  uint64_t* drain = bars + 18;
  uint64_t* p_lo = bars + 19;     // [2] slots, 128 arrivals: P of keys 0..63 in TMEM
  uint64_t* p_hi = bars + 21;     // [2] slots, 128 arrivals: P of keys 64..127
  uint64_t* o_empty = bars + 23;  // 256 arrivals: O of the piece read
  constexpr int kBars = 24;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* scan = reinterpret_cast<int*>(smem + L::kSched);  // [12] per-warp sums
  int* where = scan + 16;                                // [8] the range, found by the scan
  float2* ml = reinterpret_cast<float2*>(smem + L::kMl);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kBars; ++i) mbar_init(&bars[i], i == 23 ? 256u : i >= 19 ? 128u : (i >= 9 && i < 12) ? 2u : 1u);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  griddep_launch_dependents();
  griddep_wait();  // lengths, queries and the new cache entries; the scratch of the call before

  // ------------------------------------------------------------------ this CTA's range
  // Thread i sums the tiles of sequences i per .. i per + per - 1; a scan over the CTA gives the
  // total and finds where the range starts and where its last tile lies.
  const int units = p.n_kv * p.row_groups;
  auto tiles_of = [&](int b) { return kv_tiles(kv_end(__ldcg(p.kv_len + b), p.n_new, p.S_max)); };
  const int cta = blockIdx.x;
  int n_ctas;
  {
    const int per = (p.B + 383) / 384;
    const int b0 = threadIdx.x * per;
    int mine = 0;
    for (int b = b0; b < min(b0 + per, p.B); ++b) mine += tiles_of(b) * units;
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) scan[warp] = x;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int before = x - mine, total = 0;
#pragma unroll
    for (int w = 0; w < 12; ++w) {
      if (w < warp) before += scan[w];
      total += scan[w];
    }
    n_ctas = range_ctas(total, gridDim.x);
    const int lo = cta < n_ctas ? range_start(total, n_ctas, cta) : total;
    const int hi = cta < n_ctas ? range_start(total, n_ctas, cta + 1) : total;
    if (threadIdx.x == 0) {
      where[0] = total;
      where[1] = lo;
      where[2] = hi;
    }
    if (hi > lo && mine > 0 && lo < before + mine && hi - 1 >= before) {
      int at = before;
      for (int b = b0; b < min(b0 + per, p.B); ++b) {
        const int n = tiles_of(b) * units;
        if (lo >= at && lo < at + n) {
          where[3] = b;
          where[4] = lo - at;
        }
        if (hi - 1 >= at && hi - 1 < at + n) {  // the unit of the last tile: cut by the range's end?
          const int t = n / units, u = (hi - 1 - at) / t;
          const int u_lo = at + u * t, u_hi = u_lo + t;
          int4 d = make_int4(-1, 0, 0, 0);
          if (u_hi > hi && u_lo >= lo) d = make_int4(b, u, range_owner(total, n_ctas, u_hi - 1), 0);
          p.merge[cta] = d;
        }
        at += n;
      }
    }
    if (hi == lo && threadIdx.x == 0) p.merge[cta] = make_int4(-1, 0, 0, 0);
    if (kScores && cta == 0 && threadIdx.x == 0) *p.total_tiles = total;
    __syncthreads();
  }
  const uint32_t tmem_base = *tmem_holder;
  const int range_lo = where[1];
  KvWalk walk;
  if (where[2] > where[1])
    walk.start(where[3], where[4], tiles_of(where[3]), units, where[2] - where[1]);
  else
    walk.left = 0;

  // registers: 168 x 384 at launch >= 72 x 128 + 208 x 256
  if (warp < 4) {
    setmaxnreg_dec<72>();
    if (warp == 0) {
      if (lane == 0) {
        // ---------------------------------------------------------------- K, V producer
        const bool no_loads = p.fault && cta == 0;  // test hook: consumers wait out and abort
        int it = 0, issued_k = 0, issued_v = 0;
        bool ok = !no_loads;
        for (; ok && !walk.done(); walk.next(tiles_of)) {
          const int g = walk.u / p.row_groups;
          for (int j = walk.first; ok && j < walk.first + walk.n; ++j, ++it) {
            const int ks = it % kKS, vs = it % kVS;
            if (!(ok = mbar_wait(&k_empty[ks], ((it / kKS) & 1) ^ 1u, abort_flag, p.status))) break;
            mbar_arrive_expect_tx(&k_full[ks], L::kTile);
            uint8_t* kd = smem + L::kK + ks * L::kTile;
            tma_load_4d(kd, &tmK, &k_full[ks], 0, g, j * 128, walk.b);
            tma_load_4d(kd + L::kHalf, &tmK, &k_full[ks], 64, g, j * 128, walk.b);
            ++issued_k;
            if (!(ok = mbar_wait(&v_empty[vs], ((it / kVS) & 1) ^ 1u, abort_flag, p.status))) break;
            mbar_arrive_expect_tx(&v_full[vs], L::kTile);
            uint8_t* vd = smem + L::kV + vs * L::kTile;
            tma_load_4d(vd, &tmV, &v_full[vs], 0, g, j * 128, walk.b);
            tma_load_4d(vd + L::kHalf, &tmV, &v_full[vs], 64, g, j * 128, walk.b);
            ++issued_v;
          }
        }
        if (!no_loads) {
          // let copies still in flight land before the CTA leaves (after an abort; otherwise all
          // have been waited for)
          if (*abort_flag) {
            for (int i = max(0, issued_k - kKS); i < issued_k; ++i) mbar_wait_drain(&k_full[i % kKS], (i / kKS) & 1);
            for (int i = max(0, issued_v - kVS); i < issued_v; ++i) mbar_wait_drain(&v_full[i % kVS], (i / kVS) & 1);
          }
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------------ UMMA issuer
      // The whole warp runs the loop (its waits are warp-uniform); one elected lane issues.
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, 0, 0);   // Q, K both K-major
      constexpr uint32_t idesc_pv = idesc_bf16_f32(128, 128, 0, 1);  // P (TMEM), V MN-major
      const uint32_t q_addr = smem_u32(smem);
      const uint32_t k_addr = smem_u32(smem + L::kK);
      const uint32_t v_addr = smem_u32(smem + L::kV);
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.status));
      };
      auto commit = [&](uint64_t* bar) {
        if (elect_one_sync()) umma_commit(bar);
        __syncwarp();
      };
      int items[2] = {0, 0};  // PVs issued per slot
      uint32_t fix_par = 0;    // bit v: parity of V stage v's next v_fixed
      struct Pending {
        int slot, it;       // softmax slot, tile count
        bool fresh, fix, release, first, last;  // O starts anew; V tile fixed; V tile done; piece's first / last item
      } pend{};
      bool has_pend = false;
      int piece = 0;
      // O_i += P_i V (two halves of 64 keys as the softmax releases them)
      auto issue_pv = [&](const Pending& d) {
        const int vs = d.it % kVS;
        if (d.first && piece > 0 && !wait(o_empty, (piece - 1) & 1)) return false;
        if (!wait(&v_full[vs], (d.it / kVS) & 1)) return false;
        if (d.fix) {
          if (!wait(&v_fixed[vs], (fix_par >> vs) & 1)) return false;
          fix_par ^= 1u << vs;
        }
        const uint32_t d_o = tmem_base + 256 + d.slot * 128;
        const uint32_t a_p = tmem_base + d.slot * 128;
        const uint64_t vd = sdesc_sw128(v_addr + vs * L::kTile, L::kHalf, 1024);
        const uint32_t ph = items[d.slot] & 1;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          if (!wait(hf ? &p_hi[d.slot] : &p_lo[d.slot], ph)) return false;
          tc_fence_after();
          if (elect_one_sync()) {
#pragma unroll
            for (int kk = 4 * hf; kk < 4 * hf + 4; ++kk)
              umma_ts(d_o, a_p + kk * 8, vd + ((kk * 2048) >> 4), idesc_pv, !(d.fresh && kk == 0));
          }
          __syncwarp();
        }
        ++items[d.slot];
        if (d.release) commit(&v_empty[vs]);
        if (d.last) commit(o_full);
        return true;
      };
      bool ok = true;
      int it = 0;
      for (; ok && !walk.done(); walk.next(tiles_of), ++piece) {
        const int len = __ldcg(p.kv_len + walk.b);
        const int end = kv_end(len, p.n_new, p.S_max);
        const int safe = end < 0 ? 0 : len;  // keys below it are seen by every row
        for (int j = 0; ok && j < walk.n; ++j, ++it) {
          const bool fix = (walk.first + j + 1) * kKvTile > safe;
          if (j == 0 && !(ok = wait(q_full, piece & 1))) break;
          if (!(ok = wait(&k_full[it % kKS], (it / kKS) & 1))) break;
          tc_fence_after();
#pragma unroll
          for (int i = 0; ok && i < (kPair ? 2 : 1); ++i) {
            const int slot = kPair ? i : it & 1;
            const uint32_t d_s = tmem_base + slot * 128;
            const uint64_t qd = sdesc_sw128(q_addr + (kPair ? i : 0) * L::kTile, 0, 1024);
            const uint64_t kd = sdesc_sw128(k_addr + (it % kKS) * L::kTile, 0, 1024);
            if (elect_one_sync()) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk) {
                const uint32_t off = ((kk >> 2) * L::kHalf + (kk & 3) * 32) >> 4;
                umma_ss(d_s, qd + off, kd + off, idesc_s, kk != 0);
              }
              umma_commit(&s_full[slot]);
            }
            __syncwarp();
            const bool last_slot = !kPair || i == 1;
            if (last_slot) commit(&k_empty[it % kKS]);
            const bool last = j == walk.n - 1 && last_slot;
            if (last) commit(q_empty);
            if (has_pend && !(ok = issue_pv(pend))) break;
            pend.slot = slot;
            pend.it = it;
            pend.fresh = kPair ? j == 0 : j < 2;
            pend.fix = fix && (!kPair || i == 0);
            pend.release = last_slot;
            pend.first = j == 0 && (!kPair || i == 0);
            pend.last = last;
            has_pend = true;
          }
        }
        // the piece's last PV before the next piece's first S, which waits for its queries
        if (ok) ok = issue_pv(pend);
        has_pend = false;
      }
      if (__any_sync(0xffffffffu, *abort_flag != 0)) {  // let issued UMMAs finish before TMEM is released
        commit(drain);
        mbar_wait_drain(drain, 0);
      }
    } else if (warp == 2) {
      // ------------------------------------------------------------------ V rows nobody sees
      const int W = (p.T + 31) / 32;
      int it = 0;
      bool ok = true;
      for (; ok && !walk.done(); walk.next(tiles_of)) {
        const int len = __ldcg(p.kv_len + walk.b);
        const int end = kv_end(len, p.n_new, p.S_max);
        const int safe = end < 0 ? 0 : len;
        const int j0 = safe / kKvTile;  // first tile with a row to look at
        // drafted positions that some row sees: word w in lane w
        uint32_t seen = end < 0 ? 0u : 0xFFFFFFFFu;
        if (p.mask && end >= 0 && j0 < walk.first + walk.n) {
          const uint32_t* m = p.mask + static_cast<size_t>(walk.b) * p.T * W;
          seen = 0u;
          for (int w = 0; w < W; ++w) {
            uint32_t a = 0u;
            for (int t = lane; t < p.T; t += 32) a |= __ldcg(m + t * W + w);
            a = __reduce_or_sync(0xffffffffu, a);
            if (lane == w) seen = a;
          }
        }
        for (int j = walk.first; j < walk.first + walk.n; ++j, ++it) {
          // every tile is waited for and released, so that this warp stays in step with the ring
          const int vs = it % kVS;
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(&v_full[vs], (it / kVS) & 1, abort_flag, p.status)))) break;
          if (j < j0) {
            if (lane == 0) mbar_arrive(&v_empty[vs]);
            continue;
          }
          uint8_t* tile = smem + L::kV + vs * L::kTile;
          for (int r0 = 0; r0 < kKvTile; r0 += 32) {
            const int d = j * kKvTile + r0 + lane - safe;  // drafted index of this lane's row
            const uint32_t word = __shfl_sync(0xffffffffu, seen, (d >> 5) & 7);
            const bool dead = d >= 0 && (end < 0 || d >= p.n_new || !((word >> (d & 31)) & 1u));
            uint32_t todo = __ballot_sync(0xffffffffu, dead);
            while (todo) {  // two rows at a time, 16 lanes each (a row is 8 chunks in either half)
              const int ra = __ffs(todo) - 1;
              todo &= todo - 1;
              const int rb = todo ? __ffs(todo) - 1 : ra;
              todo &= todo - 1;
              const int r = r0 + (lane < 16 ? ra : rb), c = lane & 15;
              *reinterpret_cast<uint4*>(tile + (c >> 3) * L::kHalf + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&v_fixed[vs]);
            mbar_arrive(&v_empty[vs]);
          }
        }
      }
    } else if (lane == 0) {
      // ---------------------------------------------------------------- queries
      const bool no_loads = p.fault && cta == 0;
      int piece = 0;
      for (; !no_loads && !walk.done(); walk.next(tiles_of), ++piece) {
        if (piece > 0 && !mbar_wait(q_empty, (piece - 1) & 1, abort_flag, p.status)) break;
        const int g = walk.u / p.row_groups;
        const int t0 = (walk.u - g * p.row_groups) * (32 * L::kQTiles);
        mbar_arrive_expect_tx(q_full, L::kQTiles * L::kTile);
        for (int i = 0; i < L::kQTiles; ++i) {
          tma_load_4d(smem + i * L::kTile, &tmQ, q_full, 0, 4 * g, t0 + 32 * i, walk.b);
          tma_load_4d(smem + i * L::kTile + L::kHalf, &tmQ, q_full, 64, 4 * g, t0 + 32 * i, walk.b);
        }
      }
      if (*abort_flag && piece > 0) mbar_wait_drain(q_full, (piece - 1) & 1);
    }
  } else {
    setmaxnreg_inc<208>();
    // ------------------------------------------------------------------ softmax
    const int slot = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;  // row of the tile: position r / 4, head r & 3
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem_base + lane_off + slot * 128;
    const int W = (p.T + 31) / 32;
    const int R = p.part_rows;
    int seen_items = 0;  // of this slot
    int flat = range_lo, piece = 0;
    bool ok = true;
    for (; ok && !walk.done(); walk.next(tiles_of), ++piece) {
      const int len = __ldcg(p.kv_len + walk.b);
      const int end = kv_end(len, p.n_new, p.S_max);
      const int safe = end < 0 ? 0 : len;
      const int n_new = end < 0 ? 0 : p.n_new;
      const int g = walk.u / p.row_groups;
      const int t0 = (walk.u - g * p.row_groups) * (32 * L::kQTiles) + (kPair ? 32 * slot : 0);
      const int t = t0 + (r >> 2);
      const bool live = t < p.T;
      const bool warp_live = t0 + quarter * 8 < p.T;
      const uint32_t* mask = p.mask ? p.mask + (static_cast<size_t>(walk.b) * p.T + (live ? t : 0)) * W : nullptr;
      float m_used = -INFINITY;
      float l_sum = 0.f;
      bool fresh = true;
      for (int j = 0; j < walk.n; ++j) {
        if (!kPair && ((flat - range_lo + j) & 1) != slot) continue;
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[slot], seen_items & 1, abort_flag, p.status));
        ++seen_items;
        if (!ok) break;
        if (!warp_live) {  // rows past the last position: whatever their P is, their O is not used
          mbar_arrive(&p_lo[slot]);
          mbar_arrive(&p_hi[slot]);
          continue;
        }
        tc_fence_after();
        uint32_t sv[128];
        tmem_ld32(t_s + 0, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
        tmem_ld32(t_s + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
        tmem_ld32(t_s + 64, *reinterpret_cast<uint32_t(*)[32]>(&sv[64]));
        tmem_ld32(t_s + 96, *reinterpret_cast<uint32_t(*)[32]>(&sv[96]));
        tmem_ld_wait();
        const int key0 = (walk.first + j) * kKvTile;
        if (key0 + kKvTile > safe) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t bits = key_bits(mask, W, n_new, key0 + 32 * w - safe, live);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((bits >> i) & 1u)) sv[32 * w + i] = 0xFF800000u;  // -inf
          }
        }
        if constexpr (kScores) {
          // raw scores of the live heads, for the weights (masked keys as -inf)
          if (live) {
            float4* dst = reinterpret_cast<float4*>(p.scores + (static_cast<size_t>(flat + j) * 4 + r) * kKvTile);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              dst[i] = make_float4(__uint_as_float(sv[4 * i]), __uint_as_float(sv[4 * i + 1]),
                                   __uint_as_float(sv[4 * i + 2]), __uint_as_float(sv[4 * i + 3]));
            if (r == 0)
              p.tile_unit[flat + j] = make_int2(walk.b * units + walk.u, walk.first + j);
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
        if (fresh) {
          m_used = m_tile;
        } else if (m_tile > m_used + 8.0f) {
          grow = true;
          alpha = fast_exp2(m_used - m_tile);
          l_sum *= alpha;
          m_used = m_tile;
        }
        fresh = false;
        const float mu = (m_used == -INFINITY) ? 0.f : m_used;
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
        const float2 nmu2 = make_float2(-mu, -mu);
        float2 l4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
          for (int c = 2 * hf; c < 2 * hf + 2; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 a = ffma2(make_float2(__uint_as_float(sv[c * 32 + 2 * e]), __uint_as_float(sv[c * 32 + 2 * e + 1])),
                                     sc2, nmu2);
              const float2 pe = make_float2(fast_exp2(a.x), fast_exp2(a.y));
              l4[e & 3] = fadd2(l4[e & 3], pe);
              w[e] = pack_bf16x2(pe.x, pe.y);  // P feeds a bf16 tensor product; the sum stays fp32
            }
            tmem_st16(t_s + c * 16, w);
          }
          if (hf == 0 && __any_sync(0xffffffffu, grow)) {
            const uint32_t t_o = tmem_base + lane_off + 256 + slot * 128;
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
          mbar_arrive(hf == 0 ? &p_lo[slot] : &p_hi[slot]);
        }
        const float2 l2 = fadd2(fadd2(l4[0], l4[1]), fadd2(l4[2], l4[3]));
        l_sum += l2.x + l2.y;
      }
      // ---------------------------------------------------------------- end of a piece
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(o_full, piece & 1, abort_flag, p.status));
      if constexpr (!kPair) ml[slot * 128 + r] = make_float2(m_used, l_sum);
      // one decision for all softmax threads (and the slots' maxima and sums exchanged)
      ok = named_bar_and(1, 256, ok);
      if (!ok) break;
      tc_fence_after();
      const bool whole = walk.whole();
      const int ps = partial_slot(cta, walk.first > 0);
      float f0 = 1.f, f1 = 0.f, M = m_used, Ls = l_sum;
      if constexpr (!kPair) {
        const float2 a = ml[r], c = ml[128 + r];
        M = fmaxf(a.x, c.x);
        const float Mu = (M == -INFINITY) ? 0.f : M;
        f0 = fast_exp2(a.x - Mu);  // 0 for a slot without a tile or without a visible key
        f1 = fast_exp2(c.x - Mu);
        Ls = f0 * a.y + f1 * c.y;
      }
      const float inv = Ls > 0.f ? 1.f / Ls : (Ls == 0.f ? 0.f : Ls);  // no visible key: zeros; NaN stays
      const float scale = !whole ? 1.f : (end < 0 ? __int_as_float(0x7FC00000) : inv);
      if (warp_live) {
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.h) +
                             (static_cast<size_t>(walk.b) * p.T + (live ? t : 0)) * (p.n_kv * 512) + (g * 4 + (r & 3)) * 128;
        const int row = (kPair ? 128 * slot : 0) + r;
        float4* part = reinterpret_cast<float4*>(p.part_o) + static_cast<size_t>(ps) * 32 * R + row;
        constexpr int kChunks = kPair ? 4 : 2;  // of 32 columns
        const int c0 = kPair ? 0 : 2 * slot;
        const uint32_t t_o = tmem_base + lane_off + 256;
#pragma unroll 1
        for (int c = c0; c < c0 + kChunks; ++c) {
          float v[32];
          {
            uint32_t o0[32];
            tmem_ld32(t_o + (kPair ? 128 * slot : 0) + c * 32, o0);
            if constexpr (!kPair) {
              uint32_t o1[32];
              tmem_ld32(t_o + 128 + c * 32, o1);
              tmem_ld_wait();
              // an O that no tile of the piece wrote holds anything: left out, not multiplied by 0
#pragma unroll
              for (int i = 0; i < 32; ++i)
                v[i] = (f0 != 0.f ? f0 * __uint_as_float(o0[i]) : 0.f) + (f1 != 0.f ? f1 * __uint_as_float(o1[i]) : 0.f);
            } else {
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(o0[i]);
            }
          }
          if (!live) continue;
          if (whole) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *reinterpret_cast<uint4*>(out + c * 32 + 8 * k) = make_uint4(
                  pack_bf16x2(v[8 * k + 0] * scale, v[8 * k + 1] * scale), pack_bf16x2(v[8 * k + 2] * scale, v[8 * k + 3] * scale),
                  pack_bf16x2(v[8 * k + 4] * scale, v[8 * k + 5] * scale), pack_bf16x2(v[8 * k + 6] * scale, v[8 * k + 7] * scale));
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              part[(c * 8 + k) * R] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
          }
        }
        if (live && (kPair || slot == 0)) {
          if (!whole) p.part_ml[static_cast<size_t>(ps) * R + row] = make_float2(M, Ls);
          if constexpr (kScores) {
            if (whole) p.unit_ml[(walk.b * units + walk.u) * 4 + r] = make_float2(M, Ls);
            if (r == 0 && walk.first == 0)
              p.unit_ctas[walk.b * units + walk.u] =
                  make_int2(cta, whole ? cta : range_owner(where[0], n_ctas, flat + walk.tiles - 1));
          }
          if (end < 0 && r == 0 && walk.first == 0) atomicOr(p.status, kDevErrRange);
        }
      }
      tc_fence_before();
      mbar_arrive(o_empty);
      flat += walk.n;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// Joins the pieces of cut units: blocks (c, i) take 32 rows of the unit that CTA c began and did
// not finish.  Lane = row; warp w has columns 16 w .. 16 w + 15.  With scores, every warp then
// takes key tiles in turn and adds the four heads' weights 2^(c s - M) / l to the running sums.
template <bool kScores>
__global__ void __launch_bounds__(256) cache_finish_kernel(const CacheAttnParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_launch_dependents();
  griddep_wait();
  // after a wait that ran out the scratch may be unwritten
  if (*reinterpret_cast<volatile const int*>(p.status) & kDevErrTimeout) return;
  const int R = p.part_rows;
  const int4 d = __ldcg(p.merge + blockIdx.x);
  if (d.x >= 0) {
    const int g = d.y / p.row_groups;
    const int t0 = (d.y - g * p.row_groups) * p.group_pos;
    const int row = blockIdx.y * 32 + lane;
    const int t = t0 + (row >> 2);
    const bool live = row < 4 * p.group_pos && t < p.T;
    if (__any_sync(0xffffffffu, live)) {
      const int f = blockIdx.x, n = d.z - f + 1;
      auto slot = [&](int k) { return static_cast<size_t>(k ? partial_slot(f + k, true) : partial_slot(f, false)); };
      float M = -INFINITY;
#pragma unroll 8
      for (int k = 0; k < n; ++k) M = fmaxf(M, live ? __ldcg(p.part_ml + slot(k) * R + row).x : 0.f);
      const float Mu = M == -INFINITY ? 0.f : M;
      float l = 0.f, acc[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i] = 0.f;
      if (live) {
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
          const size_t s = slot(k);
          const float2 ml = __ldcg(p.part_ml + s * R + row);
          const float4* src = reinterpret_cast<const float4*>(p.part_o) + (s * 32 + 4 * warp) * R + row;
          float4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = __ldcg(src + static_cast<size_t>(i) * R);
          const float w = fast_exp2(ml.x - Mu);
          l += w * ml.y;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc[4 * i] += w * v[i].x;
            acc[4 * i + 1] += w * v[i].y;
            acc[4 * i + 2] += w * v[i].z;
            acc[4 * i + 3] += w * v[i].w;
          }
        }
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
        uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.h) +
                                              (static_cast<size_t>(d.x) * p.T + t) * (p.n_kv * 512) +
                                              (g * 4 + (row & 3)) * 128 + 16 * warp);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          out[i] = make_uint4(pack_bf16x2(acc[8 * i] * inv, acc[8 * i + 1] * inv),
                              pack_bf16x2(acc[8 * i + 2] * inv, acc[8 * i + 3] * inv),
                              pack_bf16x2(acc[8 * i + 4] * inv, acc[8 * i + 5] * inv),
                              pack_bf16x2(acc[8 * i + 6] * inv, acc[8 * i + 7] * inv));
      }
    }
  }
  if constexpr (kScores) {
    const int total = __ldcg(p.total_tiles);
    const int n_warps = gridDim.x * 8;
    for (int i = blockIdx.x * 8 + warp; i < total; i += n_warps) {
      const float* s = p.scores + static_cast<size_t>(i) * 4 * kKvTile;
      float x[4][4];
#pragma unroll
      for (int h = 0; h < 4; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k) x[h][k] = __ldcg(s + h * kKvTile + 32 * k + lane);
      const int2 tu = __ldcg(p.tile_unit + i);
      const int2 cs = __ldcg(p.unit_ctas + tu.x);
      float M[4], inv[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        float2 m = make_float2(-INFINITY, 0.f);
        if (cs.x == cs.y) {
          m = __ldcg(p.unit_ml + tu.x * 4 + h);
        } else {  // a cut unit: its pieces' maxima and sums, one or more pieces per lane
          for (int k = lane; k <= cs.y - cs.x; k += 32) {
            const int ps = k ? partial_slot(cs.x + k, true) : partial_slot(cs.x, false);
            const float2 o = __ldcg(p.part_ml + static_cast<size_t>(ps) * R + h);
            const float top = fmaxf(m.x, o.x), tu_ = top == -INFINITY ? 0.f : top;
            m = make_float2(top, m.y * fast_exp2(m.x - tu_) + o.y * fast_exp2(o.x - tu_));
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const float2 q = make_float2(__shfl_xor_sync(0xffffffffu, m.x, o), __shfl_xor_sync(0xffffffffu, m.y, o));
            const float top = fmaxf(m.x, q.x), tu_ = top == -INFINITY ? 0.f : top;
            m = make_float2(top, m.y * fast_exp2(m.x - tu_) + q.y * fast_exp2(q.x - tu_));
          }
        }
        M[h] = m.x == -INFINITY ? 0.f : m.x;
        inv[h] = 1.f / m.y;
      }
      float* w = p.weights + static_cast<size_t>(tu.x) * p.S_max + tu.y * kKvTile;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float a = 0.f;
        bool seen = false;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          seen |= x[h][k] != -INFINITY;  // -inf in all four: past the end (or of no weight)
          a += fast_exp2(fmaf(x[h][k], p.scale_log2, -M[h])) * inv[h];
        }
        if (seen) w[32 * k + lane] += a;
      }
    }
  }
}

}  // namespace gqa
