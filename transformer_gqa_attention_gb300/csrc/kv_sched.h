// kv_sched.h — how the attention over caches of per-sequence length shares its key tiles among
// workers.  Host and device use the same code (the host's for tests).
//
// A unit is (sequence b, kv head, group of query rows); it reads the ceil(end_b / 128) key tiles
// of its sequence (at least one, so that every unit writes its rows).  Beginning and ending a unit
// costs about as much as `cost` tiles, so each unit has that many empty places before its tiles.
// The units' places, unit after unit and sequence after sequence, form one row of `total` places, of
// which worker c of n takes places c total / n .. (c + 1) total / n - 1: equal places whatever the
// lengths are, without the host knowing them.  What a worker takes of one unit's tiles is a piece; a
// unit cut over several workers is merged from its pieces' partial results.  A worker is a CTA, a CTA
// pair, or one of a CTA's two softmax slots.
// Equal places are equal work where workers have many tiles.  A worker that starts in a unit's middle
// begins and ends its piece as well, but has no empty places for it: where most workers have one piece their
// tiles are uneven (1 to 9, 4.9 in the mean, for 6 sequences of up to 2000 keys, 150 tokens and 2 kv heads; 3
// to 9 for 8 of up to 4000 and 26 tokens; 19 to 28 for one of 32000 and 60; 210 to 219 for 32 of 8128 and 64).
#pragma once

#ifdef __CUDACC__
#define GQA_HD __host__ __device__ __forceinline__
#else
#define GQA_HD inline
#endif

namespace gqa {

constexpr int kKvTile = 128;
// Empty places per unit.  A tile takes 0.7 (pairs) to 1.5 us, the end of a unit and the start of the next
// about 3.  Measured with 2, 4, 6, 8 and 10, us: pairs 37.0, 35.5, 35.7, 35.8, 35.7 for one sequence of 32000 keys and 60
// tokens, 23.4, 20.9, 20.7, 20.4, 20.6 for 6 of up to 2000 and 150, 79.8, 69.2, 65.0, 62.8, 62.8 for a ragged batch of
// 40 units of a dozen tiles a pair; with 2, 3, 4 and 6 one tile 26.2, 25.8, 26.0, 26.3 for 8 sequences of up to 4000 and 26 tokens,
// 89.6, 89.8, 90.3, 90.8 for 32 of 4000 and 8; decode step 33.5, 34.5, 34.4, 35.5 for 16 of up to 4096 keys.
constexpr int kUnitCostPair = 8;
constexpr int kUnitCostTile = 3;
constexpr int kUnitCostDecode = 2;

// Keys that sequence b reads: its length and the n_new positions behind it; -1: out of range.
GQA_HD int kv_end(int len, int n_new, int S_max) { return len < 0 || len > S_max - n_new ? -1 : len + n_new; }

GQA_HD int kv_tiles(int end) { return end <= kKvTile ? 1 : (end + kKvTile - 1) / kKvTile; }

// Workers that share the row: no more than places, so that a unit's pieces lie with consecutive
// workers.
GQA_HD int range_workers(int total, int most) { return total < most ? total : most; }

// floor(c total / n) in 32-bit arithmetic, which holds for this many workers (a GPU has a few hundred)
constexpr int kMaxRangeWorkers = 32768;
GQA_HD int range_start(int total, int n, int c) {
  const unsigned q = static_cast<unsigned>(total) / static_cast<unsigned>(n);
  const unsigned rem = static_cast<unsigned>(total) - q * n;
  return static_cast<int>(c * q + c * rem / static_cast<unsigned>(n));
}

// The worker whose range holds place x: the last c with range_start(c) <= x.
GQA_HD int range_owner(int total, int n, int x) {
  int c = static_cast<int>(static_cast<float>(x) * static_cast<float>(n) / static_cast<float>(total));  // off by 1 or so
  c = c < n - 1 ? c : n - 1;
  while (c > 0 && range_start(total, n, c) > x) --c;
  while (c + 1 < n && range_start(total, n, c + 1) <= x) ++c;
  return c;
}

// The pieces of one range, in order.
struct KvWalk {
  int cost;       // empty places of a unit
  int b, u;       // sequence, unit in it (kv head x row groups + row group)
  int len;        // the sequence's length
  int tiles;      // key tiles of each of the sequence's units
  int first;      // the piece's first tile
  int n;          // its tiles (0: the range has no more)
  int after;      // places of the range behind the piece (0: this is the last piece)
  int lo;         // the unit's first place

  // A range of `count` places from place `begin` on, which is `offset` places into sequence b.
  GQA_HD void start(int cost_, int b_, int offset, int len_, int n_new, int S_max, int begin, int count) {
    cost = cost_;
    b = b_;
    len = len_;
    tiles = kv_tiles(kv_end(len, n_new, S_max));
    u = offset / (tiles + cost);
    const int pos = offset - u * (tiles + cost);
    lo = begin - pos;
    first = pos > cost ? pos - cost : 0;
    const int mine = min_(tiles + cost - pos, count);
    n = pos + mine - cost - first;
    if (n < 0) n = 0;
    after = rest_(count - mine);
    // (a range that ends inside the empty places has no tile of this unit, and none behind it)
  }
  GQA_HD bool done() const { return n == 0; }
  GQA_HD bool whole() const { return n == tiles; }
  // units of a sequence; len_of(b): its length
  template <typename F>
  GQA_HD void next(int units, int n_new, int S_max, F len_of) {
    n = 0;
    if (after == 0) return;
    first = 0;
    lo += tiles + cost;
    if (++u == units) {
      u = 0;
      len = len_of(++b);
      tiles = kv_tiles(kv_end(len, n_new, S_max));
    }
    const int mine = min_(tiles + cost, after);
    n = mine - cost;
    after = rest_(after - mine);
  }
  // place of the unit's tile t
  GQA_HD int place(int t) const { return lo + cost + t; }
  // number of the unit's tile t among all tiles
  GQA_HD int tile(int t, int units) const { return lo - cost * (b * units + u) + t; }

 private:
  GQA_HD static int min_(int x, int y) { return x < y ? x : y; }
  // what is left of a range, if it reaches a tile of the next unit
  GQA_HD int rest_(int x) const { return x > cost ? x : 0; }
};

// Slots of partial results: a worker has at most two pieces that are not whole units, the one its
// range starts in the middle of (slot 2c) and the one that runs on past its range (2c + 1).  The
// pieces of a cut unit are slot 2f + 1 of its first worker f and slots 2c of the workers after it.
GQA_HD int partial_slot(int worker, bool from_the_middle) { return 2 * worker + (from_the_middle ? 0 : 1); }

}  // namespace gqa
