// paged_attn.cuh — attention of one new token per sequence over a paged cache (bf16 or e4m3), split over
// the cache's length and joined.
//
//   S_h = c q_h K^T,  m_h = max S_h,  l_h = sum 2^(S_h - m_h),  O_h = sum 2^(S_h - m_h) V / l_h,  c = log2(e) / sqrt(128)
//
// The four query heads of kv head g share its keys and values, so a byte of the cache is read once for all of
// them, and reading it is what bounds the kernel: 64 sequences of 8192 keys (2.15 GB) take 306 us, 7.0 TB/s (301 where a head's
// slots lie together), 64 of up to 8192 e4m3 keys (0.54 GB) 84, one of 131000 e4m3 keys 47.  A short call is bound by
// its latencies (one sequence of 700 keys: 5.8 us): launch 1, lengths 0.7, page 0.6 and first keys 0.8 to 2, products of a
// stage 0.5, partial result and counter 1, joining 0.7.
//
// Persistent CTAs, two per SM.  All sequences' 128-key tiles form one row of places (kv_sched.h: found on the device
// from the lengths, so that one long sequence and a ragged batch both fill the GPU), cut into equal ranges; a range
// has a CTA for every kv head.  Those CTAs read the same pages at the same time, which in [page, slot, head, 128] lie
// side by side: with ranges that went over (sequence, head) pairs 64 x 8192 keys took 321 us, and e4m3 ones 189
// instead of 166.
//
//   warps 0..3  consumers: each takes a quarter of the keys of every stage; S = q K^T and O += P V with
//               mma.sync m16n8k16, rows 0..3 being the heads (4 of the 16 rows of a product that idles for two thirds
//               of the time: tcgen05's 128 rows would be emptier still); online softmax in fp32
//   warp 4      producer, three stages of 32 KB ahead: a TMA box is the largest power of two of slots that divides the
//               page (at most 64), so that a box never leaves its page.  Lane i knows the page of box i of the next 32
//               (read ahead while the boxes before are copied) and copies that box of K and of V itself.  The queries
//               come with a piece's first stage.
//
// A piece of a unit (sequence, kv head) that a CTA does not have to itself leaves an unnormalised partial
// (O, maximum m, sum l) behind; the last CTA of the unit (where they are many: of each group of them, then of the groups) to arrive
// joins the pieces in their order, so results do not depend on which one is last.
//
// Chunks of tiles taken from a counter instead of equal ranges, because the slowest CTA takes 3 to 8 % longer than the mean, cost
// more at their ends than they gained (up to 2.5 % on the largest call, 10 to 40 % lost on the others).
//
// bf16: weights enter the product with V as bf16, as in the dense cache's attention (2^-8 of each; their sum is
// taken before that): h is off by 0.0016 to 0.0020 in the 2-norm, where rounding it alone gives 0.0016 to 0.0017
// (a million keys of like weight: 0.0023).
// e4m3: numbers become fp16, which holds all of them, NaN included (bf16 would as well, but there is no
// instruction to it).  The queries are brought to fp16 with the exponent of their row's largest element taken
// out (exact down to 2^-14 of it, to 2^-25 of it below), which goes into the scale of the scores with k_scale;
// weights are 2^(c (s - m) + 15), so that they keep fp16's full precision down to 2^-29 of the largest and a million
// small ones are not lost.  v_scale is applied to the joined result.
#pragma once

#include <cuda_fp16.h>
#include <type_traits>

#include "kv_sched.h"
#include "params.h"
#include "ptx.cuh"

namespace gqa {

template <typename E>
struct PagedTile;
template <>
struct PagedTile<__nv_bfloat16> {
  static constexpr int kKeys = 64;        // of a stage
  static constexpr float kShift = 0.f;    // of the weights' exponent
};
template <>
struct PagedTile<uint8_t> {
  static constexpr int kKeys = 128;
  static constexpr float kShift = 15.f;
};

constexpr int kPagedStages = 3;
constexpr int kPagedThreads = 160;

struct PagedSmem {
  static constexpr int kHalf = 64 * 128 * 2;  // K or V of a stage: 64 keys of bf16 or 128 of e4m3
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kRed = kPagedStages * kStage;  // the consumers' results: [4 warps][4 heads][kRedRow], then (m, l)
  static constexpr int kRedRow = 136;  // floats: heads lie 8 banks apart
  static constexpr int kRedBytes = 4 * 4 * kRedRow * 4 + 4 * 4 * 8;
  static constexpr int kBar = kRed + kRedBytes;
  static constexpr int kRange = kBar + 128;
  static constexpr int kQ = kRange + 64;                // [stages] the queries of the piece that begins in the stage
  static constexpr int kQBytes = 4 * 128 * 2;
  static constexpr int kBytes = kQ + kPagedStages * kQBytes + 1024;
};

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1,
                                          __nv_bfloat16) {
  mma_bf16_16816(d, a0, 0u, a2, 0u, b0, b1);
}
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1, uint8_t) {
  mma_f16_16816(d, a0, 0u, a2, 0u, b0, b1);
}

// Four e4m3 numbers as fp16: the lower two and the upper two.
__device__ __forceinline__ void halves_of(uint32_t e4m3x4, uint32_t& lower, uint32_t& upper) {
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, u;\n\t}"
      : "=r"(lower), "=r"(upper)
      : "r"(e4m3x4));
}

// What the consumers read of a stage.  Of a 16-key block starting at key k0, keys(kk) gives the B operands of
// S += q K^T for the block's keys 0..7 and 8..15 and 16 of the 128 elements; values(i) those of O += P V
// for all 16 keys and two sets of eight columns of O.
template <typename E>
struct PagedReader;

// A box of R slots is two halves of 64 elements, [half][slot][128 bytes], 128-byte swizzle.
template <>
struct PagedReader<__nv_bfloat16> {
  uint32_t half;               // bytes from a box's first half to its second
  uint32_t k_row, v_row;       // this lane's rows, from the stage's start
  uint32_t k_swz, v_swz, k_sub, v_sub;
  __device__ __forceinline__ PagedReader(int lane, int k0, int log_box) {
    const int mi = lane >> 3;
    half = 128u << log_box;
    auto row = [&](int key) { return ((key >> log_box) << (8 + log_box)) + (key & ((1 << log_box) - 1)) * 128; };
    const int kk = k0 + (mi >> 1) * 8 + (lane & 7), kv = k0 + (mi & 1) * 8 + (lane & 7);
    k_row = row(kk);
    v_row = row(kv);
    k_swz = kk & 7;
    v_swz = kv & 7;
    k_sub = mi & 1;
    v_sub = mi >> 1;
  }
  __device__ __forceinline__ void keys(uint32_t k, int kk, uint32_t (&b)[2][2]) const {
    const uint32_t cd = 2 * kk + k_sub;
    ldsm_x4(k + k_row + (cd >> 3) * half + (((cd & 7) ^ k_swz) << 4), b[0][0], b[0][1], b[1][0], b[1][1]);
  }
  template <bool kTail>
  __device__ __forceinline__ void values(uint32_t v, int i, const uint32_t (&seen)[2], uint32_t (&b)[2][2]) const {
    const uint32_t cd = 2 * i + v_sub;
    ldsm_x4_t(v + v_row + (cd >> 3) * half + (((cd & 7) ^ v_swz) << 4), b[0][0], b[0][1], b[1][0], b[1][1]);
    if (kTail) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        b[s][0] &= seen[0];
        b[s][1] &= seen[1];
      }
    }
  }
  // the four results of a lane's sets 2 i and 2 i + 1 (of columns 16 i + c2, + 1 and 8 further on) into a head's row
  static __device__ __forceinline__ void put(float* row, int i, int c2, const float (&x)[4], const float (&y)[4]) {
    *reinterpret_cast<float2*>(row + 16 * i + c2) = make_float2(x[0], x[1]);
    *reinterpret_cast<float2*>(row + 16 * i + 8 + c2) = make_float2(y[0], y[1]);
  }
};

// A row is 128 bytes, 128-byte swizzle.  A 4-byte register of ldmatrix holds elements 4 c .. 4 c + 3 (c = lane & 3)
// of its 16: they take the places 2 c, 2 c + 1, 2 c + 8, 2 c + 9 of the product's sum, and the queries the same.
// Transposed, it holds elements 2 n, 2 n + 1 of keys 2 c and 2 c + 1: set 0 is the even elements, set 1 the odd ones.
template <>
struct PagedReader<uint8_t> {
  uint32_t row, swz, sub;
  __device__ __forceinline__ PagedReader(int lane, int k0, int) {
    const int mi = lane >> 3;
    const int key = k0 + (mi & 1) * 8 + (lane & 7);
    row = key * 128;
    swz = key & 7;
    sub = mi >> 1;
  }
  // two steps of 16 elements at once: kk even, b[step][keys 0..7, 8..15][2]
  __device__ __forceinline__ void keys2(uint32_t k, int kk, uint32_t (&b)[2][2][2]) const {
    uint32_t r[4];
    ldsm_x4(k + row + (((kk + sub) ^ swz) << 4), r[0], r[1], r[2], r[3]);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int n = 0; n < 2; ++n) halves_of(r[2 * s + n], b[s][n][0], b[s][n][1]);
  }
  template <bool kTail>
  __device__ __forceinline__ void values2(uint32_t v, int i, const uint32_t (&seen)[2], uint32_t (&b)[2][2][2]) const {
    uint32_t r[4];
    ldsm_x4_t(v + row + (((i + sub) ^ swz) << 4), r[0], r[1], r[2], r[3]);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int n = 0; n < 2; ++n) {  // keys 0..7, 8..15
        const uint32_t x = __byte_perm(kTail ? r[2 * s + n] & seen[n] : r[2 * s + n], 0u, 0x3120);
        halves_of(x, b[s][0][n], b[s][1][n]);
      }
  }
  static __device__ __forceinline__ void put(float* row, int i, int c2, const float (&x)[4], const float (&y)[4]) {
    *reinterpret_cast<float4*>(row + 16 * i + 2 * c2) = make_float4(x[0], y[0], x[1], y[1]);
  }
};

// A worker's range of the places (kv_sched.h, one unit a sequence): thread i sums those of sequences i per .. i per + per - 1;
// a scan over the CTA gives the total and finds where the share starts.
struct PagedRange {
  int* at;  // [5] per-warp sums, [7] cost; then total, workers, first place, places, sequence, offset in it, its length
  __device__ __forceinline__ int total() const { return at[8]; }
  __device__ __forceinline__ int workers() const { return at[9]; }
  __device__ __forceinline__ KvWalk walk(const PagedAttnParams& p) const {
    KvWalk w;
    w.n = 0;
    if (at[11] > 0) w.start(at[7], at[12], at[13], at[14], p.n_new, p.S_max, at[10], at[11]);
    return w;
  }
  __device__ __forceinline__ void find(const PagedAttnParams& p) const {
    constexpr int kWarps = kPagedThreads / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kMost = (1024 + kPagedThreads - 1) / kPagedThreads;  // sequences of a thread
    const int per = (p.B + kPagedThreads - 1) / kPagedThreads, b0 = threadIdx.x * per;
    int lens[kMost], places[kMost], mine = 0;
#pragma unroll
    for (int i = 0; i < kMost; ++i) lens[i] = i < per && b0 + i < p.B ? __ldcg(p.kv_len + b0 + i) : 0;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      places[i] = i < per && b0 + i < p.B ? kv_tiles(kv_end(lens[i], p.n_new, p.S_max)) + p.unit_cost : 0;
      mine += places[i];
    }
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) at[warp] = x;
    __syncthreads();
    int before = x - mine, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += at[w];
      all += at[w];
    }
    const int most = gridDim.x / p.n_kv;
    int cost = p.unit_cost;
    if (all - cost * p.B <= most) {  // every tile can have a range to itself: no places for begin and end (8 of 300 keys 7.0 -> 6.5 us)
      all -= cost * p.B;
      before -= cost * min(b0, p.B);
#pragma unroll
      for (int i = 0; i < kMost; ++i)
        if (i < per && b0 + i < p.B) places[i] -= cost;
      cost = 0;
    }
    const int n = range_workers(all, most), c = blockIdx.x / p.n_kv;
    const int lo = c < n ? range_start(all, n, c) : all, hi = c < n ? range_start(all, n, c + 1) : all;
    if (threadIdx.x == 0) {
      at[7] = cost;
      at[8] = all;
      at[9] = n;
      at[10] = lo;
      at[11] = hi - lo;
    }
    int from = before;
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      if (lo >= from && lo < from + places[i]) {
        at[12] = b0 + i;
        at[13] = lo - from;
        at[14] = lens[i];
      }
      from += places[i];
    }
    __syncthreads();
  }
};

// Keys of a piece: from its first tile to the end of its last or of the sequence.
__device__ __forceinline__ int piece_keys(const KvWalk& w, int end) {
  return max(0, min(end, (w.first + w.n) * kKvTile) - w.first * kKvTile);
}

// kGroups: units are expected to have more than 16 pieces, which are joined in groups.
template <typename E, bool kGroups>
__global__ void __launch_bounds__(kPagedThreads, 2)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ PagedAttnParams p) {
  constexpr bool k8 = sizeof(E) == 1;
  constexpr int kKeys = PagedTile<E>::kKeys;
  constexpr int kRow = 128 * sizeof(E);
  using L = PagedSmem;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* empty_bar = full_bar + kPagedStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty_bar + kPagedStages);
  volatile int* last_flag = abort_flag + 1;
  volatile int* bad_page = abort_flag + 2;  // [kPagedStages] a page of the stage's keys is out of range
  const PagedRange range{reinterpret_cast<int*>(smem + L::kRange)};

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kPagedStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  griddep_launch_dependents();
  // The lengths and a table of at most 512 KB, which the cache has pushed out of L2 since the call before, are on their
  // way there while the kernel in front ends (16 sequences of up to 4096 keys 25.3 -> 25.0 us): nothing is read yet that
  // it may still write.
  {
    const int at = blockIdx.x * kPagedThreads + threadIdx.x, table_lines = static_cast<int>((4ll * p.B * p.max_pages + 127) >> 7);
    if (at < table_lines && table_lines <= 4096) prefetch_l2(reinterpret_cast<const char*>(p.page_table) + at * 128);
    if (threadIdx.x < (4 * p.B + 127) >> 7) prefetch_l2(reinterpret_cast<const char*>(p.kv_len) + threadIdx.x * 128);
  }
  griddep_wait();  // lengths, queries and the new cache entries; the scratch of the call before
  range.find(p);
  KvWalk w = range.walk(p);
  auto len_of = [&](int b) { return __ldcg(p.kv_len + b); };
  const int g = blockIdx.x % p.n_kv;  // kv head: the CTAs of a range read the same pages at the same time

  if (warp == 4) {
    // ------------------------------------------------------------------ producer
    const int box = 1 << p.log_box;
    const int per_page = p.pool.page_size >> p.log_box;  // boxes
    const int per_stage = kKeys >> p.log_box;
    // test hook: the last worker issues no loads, so its consumers wait out and abort
    const bool no_loads = p.fault && static_cast<int>(blockIdx.x) == range.workers() * p.n_kv - 1;
    int issued = 0;
    bool ok = !no_loads;
    for (; ok && !w.done(); w.next(1, p.n_new, p.S_max, len_of)) {
      const int end = kv_end(w.len, p.n_new, p.S_max);
      const int keys = piece_keys(w, end);
      const int* table = p.page_table + static_cast<size_t>(w.b) * p.max_pages;
      const int first = w.first * (kKvTile >> p.log_box);  // box of the sequence
      const int boxes = (keys + box - 1) >> p.log_box;
      // page and slot of this lane's box of 32 boxes from `from` on
      auto look = [&](int from, int& page, int& slot) {
        const int i = from + lane;
        page = -1;
        if (i < boxes) {
          const int n = (first + i) / per_page;
          slot = (first + i - n * per_page) << p.log_box;
          page = __ldcg(table + n);
        }
      };
      int page = 0, slot = 0, next_page = 0, next_slot = 0;
      look(0, next_page, next_slot);
      for (int k0 = 0, i = 0; ok && k0 < keys; k0 += kKeys, i += per_stage, ++issued) {
        if ((i & 31) == 0) {
          page = next_page;
          slot = next_slot;
          look(i + 32, next_page, next_slot);
        }
        const int s = issued % kPagedStages;
        ok = __all_sync(0xffffffffu, mbar_wait(&empty_bar[s], ((issued / kPagedStages) & 1) ^ 1, abort_flag, p.status));
        if (!ok) break;
        const int j = lane - (i & 31);  // box of the stage
        const bool mine = j >= 0 && j < per_stage && i + j < boxes;
        const bool fits = page >= 0 && page < p.pool.n_pages;
        const uint32_t copies = __ballot_sync(0xffffffffu, mine && fits);
        const uint32_t wrong = __ballot_sync(0xffffffffu, mine && !fits);
        if (lane == 0) {
          bad_page[s] = wrong != 0;
          if (wrong) atomicOr(p.status, kDevErrRange);
          mbar_arrive_expect_tx(&full_bar[s], static_cast<uint32_t>(__popc(copies)) * 2 * box * kRow + (k0 == 0 ? L::kQBytes : 0));
          if (k0 == 0)  // the four heads' rows lie together
            bulk_load(smem + L::kQ + s * L::kQBytes,
                      static_cast<const __nv_bfloat16*>(p.q) + (static_cast<size_t>(w.b) * p.n_kv + g) * 512, L::kQBytes,
                      &full_bar[s]);
        }
        __syncwarp();
        if (mine && fits) {
          uint8_t* dst = smem + s * L::kStage + j * box * kRow;
          if constexpr (k8) {
            tma_load_4d(dst, &tmK, &full_bar[s], 0, slot, g, page);
            tma_load_4d(dst + L::kHalf, &tmV, &full_bar[s], 0, slot, g, page);
          } else {
            tma_load_5d(dst, &tmK, &full_bar[s], 0, slot, 0, g, page);
            tma_load_5d(dst + L::kHalf, &tmV, &full_bar[s], 0, slot, 0, g, page);
          }
        }
      }
    }
    if (*abort_flag) {
      for (int i = (issued > kPagedStages ? issued - kPagedStages : 0); i < issued; ++i)
        mbar_wait_drain(&full_bar[i % kPagedStages], (i / kPagedStages) & 1);
    }
    return;
  }

  // -------------------------------------------------------------------- consumers
  constexpr int kBlocks = kKeys / 64;  // 16-key blocks of a warp in a stage
  const int r0 = lane >> 2, c2 = (lane & 3) * 2;
  const bool live = r0 < 4;
  const float k_scale = k8 && p.pool.k_scale ? __ldcg(p.pool.k_scale + g) : 1.f;
  const float v_scale = k8 && p.pool.v_scale ? __ldcg(p.pool.v_scale + g) : 1.f;
  float* red_o = reinterpret_cast<float*>(smem + L::kRed);               // [4 warps][4 heads][kRedRow]
  float2* red_ml = reinterpret_cast<float2*>(red_o + 16 * L::kRedRow);  // [4 warps][4 heads]
  const PagedReader<E> rd0(lane, warp * 16 * kBlocks, p.log_box);
  int item = 0;
  for (; !w.done(); w.next(1, p.n_new, p.S_max, len_of)) {
    const int end = kv_end(w.len, p.n_new, p.S_max);
    const int keys = piece_keys(w, end);
    const bool whole = w.whole();
    const int from = whole ? 0 : range_owner(range.total(), range.workers(), w.place(0));
    const int to = whole ? 0 : range_owner(range.total(), range.workers(), w.place(w.tiles - 1));
    float scale = p.scale_log2 * k_scale;

    // A operand: rows r0 (heads), all 128 elements in the order that the keys' registers have
    uint32_t qa[8][2];
    auto queries = [&](int s) {
      const uint32_t* qw = reinterpret_cast<const uint32_t*>(smem + L::kQ + s * L::kQBytes) + (live ? r0 : 0) * 64;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const int at = k8 ? kk * 8 + c2 : kk * 8 + c2 / 2;  // pairs of elements
        qa[kk][0] = live ? qw[at] : 0u;
        qa[kk][1] = live ? qw[at + (k8 ? 1 : 4)] : 0u;
      }
      if constexpr (k8) {
        uint32_t top = 0;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
#pragma unroll
          for (int i = 0; i < 2; ++i) top = max(top, max(qa[kk][i] << 16 & 0x7F800000u, qa[kk][i] & 0x7F800000u));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        top = min(max(top, 1u << 23), 253u << 23);             // exponent field e
        const float down = __uint_as_float((254u << 23) - top);  // 2^(127 - e)
        // Kept from 0, which a key that is left out, -inf, would make NaN (a row of zeros or tiny numbers), and from infinity,
        // which would make NaN of products that are 0.  A k_scale that is no number from 0 on, or infinite, shows in the result.
        scale = scale >= 0.f && scale < INFINITY ? fminf(fmaxf(scale * __uint_as_float(top), 0x1p-126f), 0x1.fffffep127f)
                                                 : __int_as_float(0x7fc00000);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const __half2 v = __floats2half2_rn(bf16lo_to_f32(qa[kk][i]) * down, bf16hi_to_f32(qa[kk][i]) * down);
            qa[kk][i] = *reinterpret_cast<const uint32_t*>(&v);
          }
      }
    };

    float o[16][4];  // [set of eight columns]: rows r0 (0, 1) and r0 + 8 (2, 3: nothing)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m = -INFINITY, l = 0.f;  // m: largest product q k, without the scale; l: of this lane's columns

    // One stage, whose first key is k0 of the piece; kTail: keys past the last one are left out.
    auto stage = [&](auto tail, uint32_t k_addr, uint32_t v_addr, int last) {
      constexpr bool kTail = decltype(tail)::value;
      float sc[kBlocks][2][4];
#pragma unroll
      for (int blk = 0; blk < kBlocks; ++blk) {
#pragma unroll
        for (int n = 0; n < 2; ++n) sc[blk][n][0] = sc[blk][n][1] = sc[blk][n][2] = sc[blk][n][3] = 0.f;
        const uint32_t ka = k_addr + blk * 16 * kRow;  // (boxes of 16 and more slots, or rows of 128 bytes)
        if constexpr (k8) {
#pragma unroll
          for (int kk = 0; kk < 8; kk += 2) {
            uint32_t b[2][2][2];
            rd0.keys2(ka, kk, b);
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
              for (int n = 0; n < 2; ++n) mma_16816(sc[blk][n], qa[kk + s][0], qa[kk + s][1], b[s][n][0], b[s][n][1], E());
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            uint32_t b[2][2];
            rd0.keys(ka, kk, b);
#pragma unroll
            for (int n = 0; n < 2; ++n) mma_16816(sc[blk][n], qa[kk][0], qa[kk][1], b[n][0], b[n][1], E());
          }
        }
      }
      // this lane's columns are keys kb + 8 n + c2, + 1 of each block
      const int kb = warp * 16 * kBlocks;
      if (kTail) {
#pragma unroll
        for (int blk = 0; blk < kBlocks; ++blk)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (kb + blk * 16 + n * 8 + c2 + e >= last) sc[blk][n][e] = -INFINITY;
      }
      float mx = -INFINITY;
#pragma unroll
      for (int blk = 0; blk < kBlocks; ++blk)
#pragma unroll
        for (int n = 0; n < 2; ++n) mx = max3f(mx, sc[blk][n][0], sc[blk][n][1]);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // The difference to the maximum first, then its scale: the largest weight is 2^kShift exactly, and no other is above
      // it, however large the products (scaled one by one, two of 2^24 and more differ by what their rounding leaves).
      const float m_new = fmaxf(m, mx);
      const float mu = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = fast_exp2((m - mu) * scale);
      m = m_new;
      l *= alpha;
      uint32_t pa[kBlocks][2];
#pragma unroll
      for (int blk = 0; blk < kBlocks; ++blk)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float x = fast_exp2(fmaf(sc[blk][n][0] - mu, scale, PagedTile<E>::kShift));
          const float y = fast_exp2(fmaf(sc[blk][n][1] - mu, scale, PagedTile<E>::kShift));
          l += x + y;
          if constexpr (k8) {
            const __half2 v = __floats2half2_rn(x, y);
            pa[blk][n] = *reinterpret_cast<const uint32_t*>(&v);
          } else {
            pa[blk][n] = pack_bf16x2(x, y);
          }
        }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        o[i][0] *= alpha;
        o[i][1] *= alpha;
      }
#pragma unroll
      for (int blk = 0; blk < kBlocks; ++blk) {
        const uint32_t va = v_addr + blk * 16 * kRow;
        uint32_t seen[2] = {~0u, ~0u};  // of values of keys 2 c and 2 c + 1, and those 8 further on: 0 x NaN is not 0
        if (kTail) {
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int left = last - (kb + blk * 16 + n * 8 + c2);
            seen[n] = left >= 2 ? ~0u : left == 1 ? 0xFFFFu : 0u;
          }
        }
        if constexpr (k8) {
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            uint32_t b[2][2][2];
            rd0.template values2<kTail>(va, i, seen, b);
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
              for (int n = 0; n < 2; ++n) mma_16816(o[2 * (i + s) + n], pa[blk][0], pa[blk][1], b[s][n][0], b[s][n][1], E());
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t b[2][2];
            rd0.template values<kTail>(va, i, seen, b);
#pragma unroll
            for (int n = 0; n < 2; ++n) mma_16816(o[2 * i + n], pa[blk][0], pa[blk][1], b[n][0], b[n][1], E());
          }
        }
      }
    };

    bool ok = true;
    for (int k0 = 0; k0 < keys; k0 += kKeys, ++item) {
      const int s = item % kPagedStages;
      ok = __all_sync(0xffffffffu, mbar_wait(&full_bar[s], (item / kPagedStages) & 1, abort_flag, p.status));
      if (!ok) break;
      if (k0 == 0) queries(s);
      const uint32_t k_addr = smem_u32(smem + s * L::kStage), v_addr = k_addr + L::kHalf;
      if (k0 + kKeys <= keys)
        stage(std::false_type{}, k_addr, v_addr, 0);
      else
        stage(std::true_type{}, k_addr, v_addr, keys - k0);
      if (bad_page[s]) l = __int_as_float(0x7fc00000);
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty_bar[s]);
    }
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);

    // ---------------------------------------------------------- the warps' results
    if (live) {
#pragma unroll
      for (int i = 0; i < 8; ++i) PagedReader<E>::put(red_o + (warp * 4 + r0) * L::kRedRow, i, c2, o[2 * i], o[2 * i + 1]);
      if ((lane & 3) == 0) red_ml[warp * 4 + r0] = make_float2(m == -INFINITY ? m : m * scale, l);  // (no key, no scale)
    }
    // one decision for all 128 consumer threads
    if (!bar1_and_128(ok && !*abort_flag)) break;
    const int d0 = lane * 4;  // of head `warp`
    float M = -INFINITY, Ls = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int v = 0; v < 4; ++v) M = fmaxf(M, red_ml[v * 4 + warp].x);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const float2 ml = red_ml[v * 4 + warp];
      const float f = fast_exp2(ml.x - (M == -INFINITY ? 0.f : M));
      const float4 x = *reinterpret_cast<const float4*>(red_o + (v * 4 + warp) * L::kRedRow + d0);
      Ls += f * ml.y;
      acc = make_float4(acc.x + f * x.x, acc.y + f * x.y, acc.z + f * x.z, acc.w + f * x.w);
    }
    bool write = whole;
    if (!kGroups && !whole) {
      const int slot = partial_slot(blockIdx.x / p.n_kv, w.first > 0) * p.n_kv + g;
      reinterpret_cast<float4*>(p.part_o)[(static_cast<size_t>(slot) * 4 + warp) * 32 + lane] = acc;
      if (lane == 0) p.part_ml[slot * 4 + warp] = make_float2(M, Ls);
      asm volatile("bar.sync 1, 128;" ::: "memory");
      // (releases what the barrier has gathered, and acquires what the pieces before have released)
      int* counter = p.counters + w.b * p.n_kv + g;
      if (threadIdx.x == 0) *last_flag = atomic_add_acq_rel(counter, 1) == to - from;
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (*last_flag) {
        // the unit's last piece to arrive joins them, eight or sixteen pieces' loads in flight together
        write = true;
        if (threadIdx.x == 0) *counter = 0;  // ready for the next call
        M = -INFINITY;
        Ls = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        auto join = [&](auto at_once, int v0) {
          constexpr int kAtOnce = decltype(at_once)::value;
          float2 ml[kAtOnce];
          float4 x[kAtOnce];
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) {  // (past the last one: that one again)
            const int v = min(v0 + i, to);
            const size_t row = static_cast<size_t>(partial_slot(v, v > from) * p.n_kv + g) * 4 + warp;
            ml[i] = __ldcg(p.part_ml + row);
            x[i] = __ldcg(reinterpret_cast<const float4*>(p.part_o) + row * 32 + lane);
          }
          float top = M;
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) top = fmaxf(top, ml[i].x);
          const float base = top == -INFINITY ? 0.f : top;
          const float f0 = fast_exp2(M - base);
          M = top;
          Ls *= f0;
          acc = make_float4(acc.x * f0, acc.y * f0, acc.z * f0, acc.w * f0);
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i)
            if (v0 + i <= to) {
              const float f = fast_exp2(ml[i].x - base);
              Ls += f * ml[i].y;
              acc = make_float4(acc.x + f * x[i].x, acc.y + f * x[i].y, acc.z + f * x[i].z, acc.w + f * x[i].w);
            }
        };
        if (to - from < 8)
          join(std::integral_constant<int, 8>{}, from);
        else
          for (int v0 = from; v0 <= to; v0 += 16) join(std::integral_constant<int, 16>{}, v0);
      }
    }
    if (kGroups && !whole) {
      // piece i of the unit's n: where its partial result is
      const int n = to - from + 1, range_no = blockIdx.x / p.n_kv;
      auto slot = [&](int i) { return static_cast<size_t>(partial_slot(from + i, i > 0) * p.n_kv + g); };
      auto leave = [&](int i) {
        const size_t row = slot(i) * 4 + warp;
        reinterpret_cast<float4*>(p.part_o)[row * 32 + lane] = acc;
        if (lane == 0) p.part_ml[row] = make_float2(M, Ls);
      };
      leave(range_no - from);
      // More than 16 pieces are joined in groups of 8 (of more than 64: of 16), whose results take the place of their first
      // piece's, and then those.
      const int log_group = n > 64 ? 4 : n > 16 ? 3 : 0;
      int first = 0, count = n, log_step = 0;
      if (log_group) {
        first = (range_no - from) >> log_group << log_group;
        count = min(1 << log_group, n - first);
      }
      while (true) {
        asm volatile("bar.sync 1, 128;" ::: "memory");
        // (releases what the barrier has gathered, and acquires what those before have released)
        int* counter = log_group != log_step ? p.group_counters + slot(first) : p.counters + w.b * p.n_kv + g;
        if (threadIdx.x == 0) *last_flag = atomic_add_acq_rel(counter, 1) == count - 1;
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (!*last_flag) break;
        // the last one to be done joins all, eight or sixteen pieces' loads in flight together
        if (threadIdx.x == 0) *counter = 0;  // ready for the next call
        M = -INFINITY;
        Ls = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        auto join = [&](auto at_once, int i0) {
          constexpr int kAtOnce = decltype(at_once)::value;
          float2 ml[kAtOnce];
          float4 x[kAtOnce];
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) {  // (past the last one: that one again)
            const size_t row = slot(first + (min(i0 + i, count - 1) << log_step)) * 4 + warp;
            ml[i] = __ldcg(p.part_ml + row);
            x[i] = __ldcg(reinterpret_cast<const float4*>(p.part_o) + row * 32 + lane);
          }
          float top = M;
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) top = fmaxf(top, ml[i].x);
          const float base = top == -INFINITY ? 0.f : top;
          const float f0 = fast_exp2(M - base);
          M = top;
          Ls *= f0;
          acc = make_float4(acc.x * f0, acc.y * f0, acc.z * f0, acc.w * f0);
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i)
            if (i0 + i < count) {
              const float f = fast_exp2(ml[i].x - base);
              Ls += f * ml[i].y;
              acc = make_float4(acc.x + f * x[i].x, acc.y + f * x[i].y, acc.z + f * x[i].z, acc.w + f * x[i].w);
            }
        };
        if (count <= 8)
          join(std::integral_constant<int, 8>{}, 0);
        else
          for (int i0 = 0; i0 < count; i0 += 16) join(std::integral_constant<int, 16>{}, i0);
        if (log_group == log_step) {
          write = true;
          break;
        }
        __syncwarp();  // every lane has read what this overwrites
        leave(first);
        first = 0;
        count = (n + (1 << log_group) - 1) >> log_group;
        log_step = log_group;
      }
    }
    if (write) {
      float inv = 1.f / Ls, out = v_scale;  // (one after the other: v_scale / Ls may be too small for fp32)
      if (end == 0) inv = out = 0.f;
      if (end < 0) {
        inv = __int_as_float(0x7fc00000);
        if (threadIdx.x == 0) atomicOr(p.status, kDevErrRange);
      }
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.h) +
                                (static_cast<size_t>(w.b) * p.n_kv * 4 + g * 4 + warp) * 128 + d0) =
          make_uint2(pack_bf16x2(acc.x * inv * out, acc.y * inv * out), pack_bf16x2(acc.z * inv * out, acc.w * inv * out));
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");  // the results' room is free for the next piece
  }
}

}  // namespace gqa
