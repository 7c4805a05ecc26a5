// cache_roles.cuh — what the kernels of the attention over caches of per-sequence length share: the
// barriers, the search for a CTA's ranges of key tiles, the order in which its roles walk them, and
// the roles that do not depend on how the products are laid out (TMA producers, and the warp that
// clears V rows which nobody sees).
//
// Warps of a CTA (384 threads):
//   warp 0      TMA producer of the 128-key K tiles, running ahead over the ends of units
//   warp 1      TMEM owner and UMMA issuer
//   warp 2      zeroes the rows of a V tile that no row sees (past the end of the sequence, or
//               drafted positions that nobody's mask names): their weight is 0, but 0 x NaN is not
//   warp 3      TMA producer of the V tiles (a tile's V is needed a softmax later than its K) and
//               of each unit's queries, once the last S of the unit before has read its own
//   warps 4..11 softmax
// Which products they work on is the kernel's mode:
//   kTwoWorkers  warps 4..7 and 8..11 are workers of their own (kv_sched.h), each with its own range
//                of tiles, queries, S and O (cache_decode.cuh)
//   kOneTile     one worker: S alternates between two buffers from tile to tile, queries and O from
//                piece to piece (cache_attn.cuh)
#pragma once

#include <type_traits>

#include "kv_sched.h"
#include "params.h"
#include "ptx.cuh"

namespace gqa {

enum CacheMode : int { kTwoWorkers, kOneTile };
constexpr int mode_workers(int mode) { return mode == kTwoWorkers ? 2 : 1; }

// Buffer (0 or 1) that queries and O of piece `piece` take, and how many pieces had it before.
template <int kMode>
__device__ __forceinline__ int piece_buffer(int worker, int piece) {
  return kMode == kTwoWorkers ? worker : piece & 1;
}
template <int kMode>
__device__ __forceinline__ int piece_turn(int piece) {
  return kMode == kOneTile ? piece >> 1 : piece;
}

constexpr int kKvTileBytes = kKvTile * 128 * 2;  // 128 keys x 128 bf16, two 64-column halves
constexpr int kKvHalfBytes = kKvTileBytes / 2;
constexpr int kKStages = 2;
constexpr int kVStages = 3;

struct CacheBars {
  static constexpr int kCount = 28;
  static constexpr int kBytes = 256;  // barriers, TMEM address, abort flag
  uint64_t* bars;
  __device__ __forceinline__ explicit CacheBars(uint8_t* at) : bars(reinterpret_cast<uint64_t*>(at)) {}
  __device__ __forceinline__ uint64_t* q_full(int slot) const { return bars + slot; }
  __device__ __forceinline__ uint64_t* q_empty(int slot) const { return bars + 2 + slot; }
  __device__ __forceinline__ uint64_t* k_full(int stage) const { return bars + 4 + stage; }
  __device__ __forceinline__ uint64_t* k_empty(int stage) const { return bars + 6 + stage; }
  __device__ __forceinline__ uint64_t* v_full(int stage) const { return bars + 8 + stage; }
  __device__ __forceinline__ uint64_t* v_fixed(int stage) const { return bars + 11 + stage; }
  __device__ __forceinline__ uint64_t* s_full(int slot) const { return bars + 14 + slot; }
  __device__ __forceinline__ uint64_t* o_full(int slot) const { return bars + 16 + slot; }
  __device__ __forceinline__ uint64_t* drain() const { return bars + 18; }
  // 2 arrivals: the PV that used the tile, and warp 2
  __device__ __forceinline__ uint64_t* v_empty(int stage) const { return bars + 19 + stage; }
  // arrivals of its writers: P of the tile's first and second 64 keys (or of all of them: lo)
  __device__ __forceinline__ uint64_t* p_lo(int slot) const { return bars + 22 + slot; }
  __device__ __forceinline__ uint64_t* p_hi(int slot) const { return bars + 24 + slot; }
  // arrivals of those that read O
  __device__ __forceinline__ uint64_t* o_empty(int slot) const { return bars + 26 + slot; }
  __device__ __forceinline__ uint32_t* tmem_holder() const { return reinterpret_cast<uint32_t*>(bars + kCount); }
  __device__ __forceinline__ volatile int* abort_flag() const { return reinterpret_cast<volatile int*>(tmem_holder() + 1); }
  __device__ __forceinline__ void init(uint32_t p_writers, uint32_t o_readers) const {
    for (int i = 0; i < kCount; ++i) mbar_init(&bars[i], i < 19 ? 1u : i < 22 ? 2u : i < 26 ? p_writers : o_readers);
    *abort_flag() = 0;
    fence_mbar_init();
  }
};

// The CTA's ranges of places (kv_sched.h), in shared memory: thread i sums the places of sequences i
// per .. i per + per - 1 (B <= 1024: per <= 3); a scan over the CTA gives the total and finds where the
// ranges start.  Called by all 384 threads.
struct CacheRanges {
  static constexpr int kBytes = 128;
  int* scan;   // [12] per-warp sums
  int* where;  // total, workers, then per worker: first place, places, sequence, offset in it, its length

  __device__ __forceinline__ explicit CacheRanges(uint8_t* at) : scan(reinterpret_cast<int*>(at)), where(scan + 16) {}
  __device__ __forceinline__ int total() const { return where[0]; }
  __device__ __forceinline__ int workers() const { return where[1]; }
  __device__ __forceinline__ KvWalk walk(int s, const CacheAttnParams& p) const {
    KvWalk w;
    w.n = 0;
    if (where[3 + 5 * s] > 0)
      w.start(p.unit_cost, where[4 + 5 * s], where[5 + 5 * s], where[6 + 5 * s], p.n_new, p.S_max, where[2 + 5 * s], where[3 + 5 * s]);
    return w;
  }

  // of kWork workers from `first` on, `most` in all
  template <int kWork>
  __device__ __forceinline__ void find(const CacheAttnParams& p, int first, int most) const {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int units = p.n_kv * p.row_groups;
    const int per = (p.B + 383) / 384;
    const int b0 = threadIdx.x * per;
    int lens[3], places[3], mine = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const bool in = i < per && b0 + i < p.B;
      lens[i] = in ? __ldcg(p.kv_len + b0 + i) : 0;
      places[i] = in ? (kv_tiles(kv_end(lens[i], p.n_new, p.S_max)) + p.unit_cost) * units : 0;
      mine += places[i];
    }
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    int before = x - mine, total = 0;
#pragma unroll
    for (int w = 0; w < 12; ++w) {
      if (w < warp) before += scan[w];
      total += scan[w];
    }
    const int n_work = range_workers(total, most);
    if (threadIdx.x == 0) {
      where[0] = total;
      where[1] = n_work;
      if (p.total_tiles && blockIdx.x == 0) *p.total_tiles = total - p.unit_cost * units * p.B;
    }
#pragma unroll
    for (int s = 0; s < kWork; ++s) {
      const int v = first + s;
      const int lo = v < n_work ? range_start(total, n_work, v) : total;
      const int hi = v < n_work ? range_start(total, n_work, v + 1) : total;
      if (threadIdx.x == 0) {
        where[2 + 5 * s] = lo;
        where[3 + 5 * s] = hi - lo;
      }
      int at = before;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        if (lo >= at && lo < at + places[i]) {
          where[4 + 5 * s] = b0 + i;
          where[5 + 5 * s] = lo - at;
          where[6 + 5 * s] = lens[i];
        }
        at += places[i];
      }
    }
    __syncthreads();
  }
};

// One worker's place in its range.
struct CacheLane {
  KvWalk w;
  int j, piece;  // tile inside the piece, piece
};

// A CTA's tiles in the order in which every role takes them: the workers in turn.
template <int kWork>
struct CacheTiles {
  const CacheAttnParams& p;
  CacheLane l0, l1;
  __device__ __forceinline__ CacheTiles(const CacheAttnParams& p_, const CacheRanges& r)
      : p(p_), l0{r.walk(0, p_), 0, 0}, l1{r.walk(kWork - 1, p_), 0, 0} {}
  __device__ __forceinline__ void advance(CacheLane& l) {
    if (++l.j == l.w.n) {
      l.j = 0;
      ++l.piece;
      l.w.next(p.n_kv * p.row_groups, p.n_new, p.S_max, [&](int b) { return __ldcg(p.kv_len + b); });
    }
  }
  // step(slot constant, lane) -> go on; false if a step gave up
  template <typename F>
  __device__ __forceinline__ bool each(F step) {
    while (true) {
      const bool d0 = l0.w.done(), d1 = kWork == 1 || l1.w.done();
      if (d0 && d1) return true;
      if (!d0) {
        if (!step(std::integral_constant<int, 0>{}, l0)) return false;
        advance(l0);
      }
      if (!d1) {
        if (!step(std::integral_constant<int, 1>{}, l1)) return false;
        advance(l1);
      }
    }
  }
};

// K and V are read once, unless a sequence has several groups of rows: they leave L2 first, which
// keeps the partial results, the scores and the kernel's own code there.
__device__ __forceinline__ uint64_t kv_policy(const CacheAttnParams& p) { return l2_policy(p.row_groups == 1); }

// Lane 0 of warp 0.
template <int kWork>
__device__ __forceinline__ void produce_k(const CacheAttnParams& p, const CacheRanges& ranges, const CacheBars& bar,
                                          const CUtensorMap* tmK, uint8_t* ring) {
  CacheTiles<kWork> tiles(p, ranges);
  volatile int* abort_flag = bar.abort_flag();
  const uint64_t policy = kv_policy(p);
  int it = 0;
  tiles.each([&](auto, CacheLane& l) {
    const int st = it % kKStages;
    if (!mbar_wait(bar.k_empty(st), ((it / kKStages) & 1) ^ 1u, abort_flag, p.status)) return false;
    mbar_arrive_expect_tx(bar.k_full(st), kKvTileBytes);
    uint8_t* dst = ring + st * kKvTileBytes;
    const int g = l.w.u / p.row_groups, key0 = (l.w.first + l.j) * kKvTile;
    tma_load_4d_hint(dst, tmK, bar.k_full(st), 0, g, key0, l.w.b, policy);
    tma_load_4d_hint(dst + kKvHalfBytes, tmK, bar.k_full(st), 64, g, key0, l.w.b, policy);
    ++it;
    return true;
  });
  if (*abort_flag)  // let copies still in flight land before the CTA leaves
    for (int i = max(0, it - kKStages); i < it; ++i) mbar_wait_drain(bar.k_full(i % kKStages), (i / kKStages) & 1);
}

// Lane 0 of warp 3.  A unit's queries are q_rows rows (positions x 4 heads; the box of tmQ) in two
// halves of 64 columns, q_half bytes apart.
template <int kMode>
__device__ __forceinline__ void produce_vq(const CacheAttnParams& p, const CacheRanges& ranges, const CacheBars& bar,
                                           const CUtensorMap* tmQ, const CUtensorMap* tmV, uint8_t* q, int q_rows,
                                           int q_half, uint8_t* ring) {
  CacheTiles<mode_workers(kMode)> tiles(p, ranges);
  volatile int* abort_flag = bar.abort_flag();
  const uint64_t policy = kv_policy(p);
  int it = 0, asked = 0;  // queries asked for: buffer 0 in the low half, 1 in the high
  tiles.each([&](auto S, CacheLane& l) {
    const int g = l.w.u / p.row_groups;
    if (l.j == 0) {
      const int t0 = (l.w.u - g * p.row_groups) * p.group_pos;
      const int at = piece_buffer<kMode>(S.value, l.piece), turn = piece_turn<kMode>(l.piece);
      if (turn > 0 && !mbar_wait(bar.q_empty(at), (turn - 1) & 1, abort_flag, p.status)) return false;
      mbar_arrive_expect_tx(bar.q_full(at), q_rows * 256);
      uint8_t* dst = q + at * 2 * q_half;
      tma_load_4d(dst, tmQ, bar.q_full(at), 0, 4 * g, t0, l.w.b);
      tma_load_4d(dst + q_half, tmQ, bar.q_full(at), 64, 4 * g, t0, l.w.b);
      asked += at ? 0x10000 : 1;
    }
    const int st = it % kVStages;
    if (!mbar_wait(bar.v_empty(st), ((it / kVStages) & 1) ^ 1u, abort_flag, p.status)) return false;
    mbar_arrive_expect_tx(bar.v_full(st), kKvTileBytes);
    uint8_t* dst = ring + st * kKvTileBytes;
    const int key0 = (l.w.first + l.j) * kKvTile;
    tma_load_4d_hint(dst, tmV, bar.v_full(st), 0, g, key0, l.w.b, policy);
    tma_load_4d_hint(dst + kKvHalfBytes, tmV, bar.v_full(st), 64, g, key0, l.w.b, policy);
    ++it;
    return true;
  });
  if (*abort_flag) {
    for (int i = max(0, it - kVStages); i < it; ++i) mbar_wait_drain(bar.v_full(i % kVStages), (i / kVStages) & 1);
    if (asked & 0xFFFF) mbar_wait_drain(bar.q_full(0), ((asked & 0xFFFF) - 1) & 1);
    if (asked >> 16) mbar_wait_drain(bar.q_full(1), ((asked >> 16) - 1) & 1);
  }
}

// Keys of the sequence that every row sees (a length out of range: none).
__device__ __forceinline__ int keys_all_see(const CacheAttnParams& p, int len) {
  return kv_end(len, p.n_new, p.S_max) < 0 ? 0 : len;
}

// The unit of a worker's last piece as the merge wants it (CacheAttnParams::merge): whether it goes
// on past the worker's range.
__device__ __forceinline__ int4 goes_on(const CacheRanges& ranges, const KvWalk& w, int worker) {
  if (w.first + w.n == w.tiles) return make_int4(-1, 0, 0, 0);
  return make_int4(w.b, w.u, w.first > 0 ? range_owner(ranges.total(), ranges.workers(), w.place(0)) : worker,
                   range_owner(ranges.total(), ranges.workers(), w.place(w.tiles - 1)));
}

// Which rows of a V tile no row of the product sees; used by a whole warp.
struct ClearRows {
  int seen_b = -1;
  uint32_t seen = 0;  // drafted positions of sequence seen_b that some row sees: word i in lane i
  // Whether the tile reaches past the keys that every row sees.
  __device__ __forceinline__ bool prepare(const CacheAttnParams& p, const CacheLane& l) {
    if ((l.w.first + l.j + 1) * kKvTile <= keys_all_see(p, l.w.len)) return false;
    if (seen_b != l.w.b) {
      const int lane = threadIdx.x & 31;
      const int W = (p.T + 31) / 32;
      seen_b = l.w.b;
      seen = 0xFFFFFFFFu;
      if (p.mask && kv_end(l.w.len, p.n_new, p.S_max) >= 0) {
        const uint32_t* m = p.mask + static_cast<size_t>(seen_b) * p.T * W;
        seen = 0u;
        for (int i = 0; i < W; ++i) {
          uint32_t a = 0u;
          for (int t = lane; t < p.T; t += 32) a |= __ldcg(m + t * W + i);
          a = __reduce_or_sync(0xffffffffu, a);
          if (lane == i) seen = a;
        }
      }
    }
    return true;
  }
  // Zeroes them: a lane takes a row, at(row, c) is the address of its 16-byte chunk c < kChunks.  Whether
  // there was such a row.
  template <int kChunks, typename F>
  __device__ __forceinline__ bool rows(const CacheAttnParams& p, const CacheLane& l, F at) const {
    const int lane = threadIdx.x & 31;
    const bool bad = kv_end(l.w.len, p.n_new, p.S_max) < 0;
    const int d0 = (l.w.first + l.j) * kKvTile - keys_all_see(p, l.w.len);  // drafted index of row 0
    bool any = false;
#pragma unroll
    for (int r0 = 0; r0 < kKvTile; r0 += 32) {
      const int d = d0 + r0 + lane;
      const uint32_t word = __shfl_sync(0xffffffffu, seen, (d >> 5) & 7);
      const bool dead = d >= 0 && (bad || d >= p.n_new || !((word >> (d & 31)) & 1u));
      any |= dead;
      if (dead) {
#pragma unroll
        for (int k = 0; k < kChunks; ++k)  // (eight lanes at a time: in other banks)
          *reinterpret_cast<uint4*>(at(r0 + lane, (k + lane) % kChunks)) = make_uint4(0, 0, 0, 0);
      }
    }
    return __any_sync(0xffffffffu, any);
  }
};

// Whole warp 2.  Also publishes, for the merge, the unit that goes on past each worker's range.
template <int kWork>
__device__ __forceinline__ void clear_v(const CacheAttnParams& p, const CacheRanges& ranges, const CacheBars& bar,
                                        uint8_t* ring) {
  CacheTiles<kWork> tiles(p, ranges);
  volatile int* abort_flag = bar.abort_flag();
  const int lane = threadIdx.x & 31;
  ClearRows clear;
  int it = 0;
  if (lane == 0) {  // workers without a tile
    if (tiles.l0.w.done()) p.merge[kWork * blockIdx.x] = make_int4(-1, 0, 0, 0);
    if (kWork == 2 && tiles.l1.w.done()) p.merge[kWork * blockIdx.x + 1] = make_int4(-1, 0, 0, 0);
  }
  tiles.each([&](auto S, CacheLane& l) {
    const int worker = kWork * blockIdx.x + S.value;
    if (lane == 0 && l.j == 0 && l.w.after == 0) p.merge[worker] = goes_on(ranges, l.w, worker);
    const bool fix = clear.prepare(p, l);
    // every tile is waited for and released, so that this warp stays in step with the ring
    const int st = it % kVStages;
    if (!__all_sync(0xffffffffu, mbar_wait(bar.v_full(st), (it / kVStages) & 1, abort_flag, p.status))) return false;
    if (fix) {
      clear.rows<16>(p, l, [&](int r, int c) {
        return ring + st * kKvTileBytes + (c >> 3) * kKvHalfBytes + r * 128 + (c & 7) * 16;
      });
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar.v_fixed(st));
    }
    if (lane == 0) mbar_arrive(bar.v_empty(st));
    ++it;
    return true;
  });
}

// The whole of warp 1.  In turn for each tile: S (issue_s), then the PV of the tile before
// (issue_pv_mma), so that the tensor core works while a softmax runs.
//   issue_s(S buffer, query buffer, K stage): the UMMAs of S
//   issue_pv_mma(S buffer, O buffer, V stage, half, first): those of O += P V for keys 64 half .. + 63
//   (kHalves = 2) or all keys (kHalves = 1), O anew if first
template <int kMode, int kHalves, typename FS, typename FP>
__device__ __forceinline__ void issue_all(const CacheAttnParams& p, const CacheRanges& ranges, const CacheBars& bar,
                                          FS issue_s, FP issue_pv_mma) {
  CacheTiles<mode_workers(kMode)> tiles(p, ranges);
  volatile int* abort_flag = bar.abort_flag();
  auto wait = [&](uint64_t* b, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(b, parity, abort_flag, p.status));
  };
  uint32_t fix_par = 0;  // bit v: parity of V stage v's next v_fixed
  uint32_t p_par = 0;    // bit i: parity of S buffer i's next P
  struct Pending {
    int slot, o, turn, it;           // S and O buffer, pieces that had the O before, tile count
    bool first, last, fix;           // first / last tile of the piece; V tile to be cleared
  } pend{};
  bool has_pend = false;
  auto issue_pv = [&] {
    const Pending d = pend;
    has_pend = false;
    const int vs = d.it % kVStages;
    // a new O takes the place of an earlier piece's
    if (d.first && d.turn > 0 && !wait(bar.o_empty(d.o), (d.turn - 1) & 1)) return false;
    if (!wait(bar.v_full(vs), (d.it / kVStages) & 1)) return false;
    if (d.fix) {
      if (!wait(bar.v_fixed(vs), (fix_par >> vs) & 1)) return false;
      fix_par ^= 1u << vs;
    }
    const uint32_t ph = (p_par >> d.slot) & 1;
    p_par ^= 1u << d.slot;
#pragma unroll
    for (int hf = 0; hf < kHalves; ++hf) {
      if (!wait(hf ? bar.p_hi(d.slot) : bar.p_lo(d.slot), ph)) return false;
      tc_fence_after();
      if (elect_one_sync()) {
        issue_pv_mma(d.slot, d.o, vs, hf, d.first);
        if (hf == kHalves - 1) {
          umma_commit(bar.v_empty(vs));
          if (d.last) umma_commit(bar.o_full(d.o));
        }
      }
      __syncwarp();
    }
    return true;
  };
  int it = 0;
  const bool ok = tiles.each([&](auto S, CacheLane& l) {
    const bool fix = (l.w.first + l.j + 1) * kKvTile > keys_all_see(p, l.w.len);
    const bool first = l.j == 0, last = l.j == l.w.n - 1;
    const int ks = it % kKStages;
    const int turn = piece_turn<kMode>(l.piece);
    const int slot = kMode == kTwoWorkers ? S.value : it & 1;
    const int at = piece_buffer<kMode>(S.value, l.piece);
    // P of the buffer's last tile is used up before the softmax of S takes its place (the other
    // worker has no more tiles in between)
    if (kMode == kTwoWorkers && has_pend && pend.slot == slot && !issue_pv()) return false;
    if (first && !wait(bar.q_full(at), turn & 1)) return false;
    if (!wait(bar.k_full(ks), (it / kKStages) & 1)) return false;
    tc_fence_after();
    if (elect_one_sync()) {
      issue_s(slot, at, ks);
      umma_commit(bar.s_full(slot));
      umma_commit(bar.k_empty(ks));
      if (last) umma_commit(bar.q_empty(at));
    }
    __syncwarp();
    if (has_pend && !issue_pv()) return false;
    pend = Pending{slot, at, turn, it, first, last, fix};
    has_pend = true;
    ++it;
    return true;
  });
  if (ok && has_pend) issue_pv();
  if (__any_sync(0xffffffffu, *abort_flag != 0)) {  // let issued UMMAs finish before TMEM is released
    if (elect_one_sync()) umma_commit(bar.drain());
    __syncwarp();
    mbar_wait_drain(bar.drain(), 0);
  }
}

// Visibility of 32 N keys to one row, whose first has drafted index `base` (negative: prefix, always seen),
// over n_new drafted positions: the mask row's N + 1 words around them, loaded ahead of their use.  A row
// without a mask (null) that is live sees all n_new.
template <int N>
struct KeyWords {
  uint32_t w[N + 1];
  int base;
  __device__ __forceinline__ void load(const uint32_t* mask, int W, int base_, bool live) {
    base = base_;
    const int q = base >> 5;  // floor
#pragma unroll
    for (int i = 0; i <= N; ++i) {
      // (without conditions, so that all are in flight together)
      const uint32_t word = mask ? __ldcg(mask + min(max(q + i, 0), W - 1)) : 0xFFFFFFFFu;
      w[i] = q + i < 0 ? 0xFFFFFFFFu : q + i < W && live ? word : 0u;
    }
  }
  // of keys 32 c .. 32 c + 31
  __device__ __forceinline__ uint32_t bits(int c, int n_new) const {
    const uint32_t x = __funnelshift_r(w[c], w[c + 1], base & 31);
    const int rem = n_new - (base + 32 * c);
    return rem <= 0 ? 0u : rem < 32 ? x & ((1u << rem) - 1u) : x;
  }
};

}  // namespace gqa
