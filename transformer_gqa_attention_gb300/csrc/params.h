// params.h — launch parameter blocks and constants shared by the kernels and the host
// code (no device code here).
#pragma once

#include <vector_types.h>

#include <cstdint>
#include <type_traits>

#include "gqa_attn.h"

namespace gqa {

// Status bits OR-ed into the context's device status word.
constexpr int kDevErrTimeout = 1;
constexpr int kDevErrRange = 2;  // a per-sequence length or path read on the device is out of range

// Upper bound for any single device-side wait (wall-clock, via %globaltimer).
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s
constexpr uint64_t kDrainLimitNs = 200000000ull;  // 0.2 s while draining after an abort

// kQkvRope / kStoreF32: many-token epilogues.  kSplitKQkv / kSplitKOut: the same two
// epilogues after the cluster-wide split-K reduction of the few-token kernel.  kQkvRopeSeq /
// kSplitKQkvSeq: the Q/K/V ones with a start of its own for every sequence.
enum EpiMode : int { kQkvRope = 0, kStoreF32 = 1, kSplitKQkv = 3, kSplitKOut = 4, kQkvRopeSeq = 5, kSplitKQkvSeq = 6 };

struct GemmParams {
  int M, N;          // rows of A, rows of B
  int num_kb;        // K / 64
  int splits;        // few-token kernel: k splits = cluster size
  int n_tiles;       // CTA-pair kernels: 256-wide output tiles along N (split-K kernels: 1)
  int m_tiles;       // ceil(M / 128)
  // CTA-pair kernel schedule: full_rounds rounds of whole 256x256 tiles, then the tiles of
  // the last, partial round cut into pieces of tail_w columns (0: whole tiles throughout)
  int full_rounds, tail_w;
  // Q/K/V epilogues: the packed weight's rows are q_cols query features (4 heads x 128 per
  // kv group), then kv_cols key and kv_cols value features (128 per kv group); Q_r rows are
  // q_cols wide and a cache position holds kv_cols features.  The whole block: 4096 / 1024.
  int q_cols, kv_cols;
  // epilogue operands
  void* out0;        // kQkvRope: Q_r [M,q_cols] bf16 | kStoreF32: D fp32
  void* out1;        // kQkvRope: cache_k
  void* out2;        // kQkvRope: cache_v
  const float* R;    // Q/K/V epilogues: [T,64,2] (kQkvRopeSeq, kSplitKQkvSeq: [tokens,64,2])
  int T, S_max, start_pos;
  int ldo;           // kStoreF32: row stride (floats)
  void* fin0;        // split-K final outputs: Q_r [N,q_cols] bf16 | Delta [N,4096] fp32
  void* fin1;        // kSplitKQkv: cache_k
  void* fin2;        // kSplitKQkv: cache_v
  int* status;
  int fault;         // test hook: the first work unit's producer issues no loads (its waits run out)
  // residual form of the block (both null for the block alone)
  const float* row_scale;  // Q/K/V epilogues: 1 / rms of each token row (attention_norm)
  const void* residual;    // Delta epilogues: x [tokens, 4096] bf16, added to Delta
};

static_assert(sizeof(GemmParams) <= 144, "eight bytes more take 16-token steps 0.2 to 0.3 us of 32 to 78");

// Of kQkvRopeSeq and kSplitKQkvSeq, so that the other projections' parameters stay as short as they are.
struct GemmSeqParams : GemmParams {
  // first position of each sequence [B] (device), read in place of start_pos; a sequence whose T positions
  // do not fit the cache is not written
  const int* seq_start;
};
template <int EPI>
using EpiParams = std::conditional_t<EPI == kQkvRopeSeq || EPI == kSplitKQkvSeq, GemmSeqParams, GemmParams>;

struct FlashParams {
  int B, T, S_max, start_pos, causal;
  int n_kv;             // kv groups (heads of K/V) of the context; 4 query heads each
  int n_qtiles;
  int groups_per_band;  // (sequence, kv group) pairs scheduled together (divides n_kv B)
  int* status;
  int fault;  // test hook: CTA 0's producer issues no loads (its waits run out)
  float scale_log2;  // log2(e) / sqrt(128)
};

constexpr int kDecStages = 3;
constexpr int kDecTileKeys = 64;

struct DecodeParams {
  int B, kv_len, n_splits, tiles_per_split;
  int n_kv;       // kv groups of the context (4 query heads each; q and H rows are 512 n_kv wide)
  // query positions: T per sequence, the first at absolute position q_start (decode: T = 1,
  // q_start = kv_len - 1); with causal, query t sees keys 0 .. q_start + t, else all kv_len
  int T, q_start, causal;
  int n_pg;       // position groups per sequence (ceil(T / positions per CTA))
  const void* q;  // [B, T, 512 n_kv] bf16 rotated queries
  float* part_o;           // [B, n_kv, n_pg, n_splits, rows, 128]
  float* part_ml;          // [B, n_kv, n_pg, n_splits, rows, 2]
  int* counters;           // [B*n_kv*n_pg] arrival counters: the last split merges (null: separate merge kernel)
  void* H;        // [B, T, 512 n_kv] bf16 (combine output)
  int* status;
  // decode_combine_kernel only: when *status is non-zero (a split of this call gave up a
  // wait), H is written as NaN and the status bits are OR-ed into *status_sticky (null: not)
  int* status_sticky;
  int fault;      // test hook: CTA (0, 0, 0)'s producer issues no loads (its waits run out)
  float scale_log2;
};

// At most this many positions run on one 128-row tile (positions x 4 heads), more on the two tiles of a
// CTA pair, which a few positions leave half empty: at T = 8, 26 and 32, us, 32 sequences of 4000 keys take
// 89, 92, 95 on one tile and 95, 99, 101 on a pair; 8 of 4000 30.9, 34.9, 35.3 and 34.1, 35.7, 36.2; one of 8000
// 16.3, 18.2, 18.7 and 16.4, 17.6, 18.0; one of 300 10.1, 11.8, 12.1 and 10.9, 11.8, 12.0.
constexpr int kOneTilePos = 32;

// Attention of a few positions per sequence over caches of per-sequence length (tree attention,
// decode attention that accumulates key weights).  Row t of sequence b sees keys 0 ..
// kv_len[b] - 1 and, of the n_new keys behind them, those whose bit is set in mask[b, t].
struct CacheAttnParams {
  int B, T, S_max;
  int n_kv;                // kv groups of the context (4 query heads each; q and h rows are 512 n_kv wide)
  int n_new;               // keys behind kv_len[b] (the call's own positions; at most T)
  const uint32_t* mask;    // [B, T, ceil(T / 32)] visibility bits of the n_new keys; null: all visible
  const int* kv_len;       // [B]
  void* h;                 // [B, T, 512 n_kv] bf16
  float* weights;          // [B, n_kv, S_max] accumulated key weights (T = 1), or null
  int* status;
  int fault;               // test hook: the last worker issues no loads (its waits run out)
  float scale_log2;        // log2(e) / sqrt(128)
  // rows: a kv head's T positions in row_groups groups of group_pos (kOneTilePos, or 64 on two tiles)
  int row_groups, group_pos;
  int unit_cost;           // empty places of a unit in the workers' shares (kv_sched.h)
  // scratch: per worker the unit that goes on past its range (sequence or -1, unit, the unit's first
  // and last worker), the partial results of cut units ([2 workers][32 float4 columns][part_rows], with
  // weights [2 workers][part_rows][128]) and their (maximum, sum)
  int4* merge;
  float* part_o;
  float2* part_ml;
  int part_rows;
  // with weights: scores [tile][128 keys][4 heads], each tile's (unit, index in it, the unit's first
  // and last worker) and, for whole units, each head's (maximum, sum)
  float* scores;
  int4* tile_unit;
  float2* unit_ml;
  int* total_tiles;
};

// The accepted path of each sequence moved to the front of its drafted positions.
struct CommitParams {
  int B, S_max, T, n_kv;
  void* k;
  void* v;
  const int* prefix_len;  // [B]
  const int* path;        // [B, T]
  const int* n_accept;    // [B]
  int* new_len;           // [B], may be prefix_len
  int* status;
};

// Selection and move of the cache positions that an eviction keeps.
struct EvictParams {
  int B, S_max, S_out, n_kv;
  int budget, n_first, n_recent;
  int in_place;
  const void* k;
  const void* v;
  const float* weights;   // [B, n_kv, S_max]
  const int* kv_len;      // [B]
  void* out_k;            // [B, S_out, n_kv, 128]
  void* out_v;
  float* out_weights;     // [B, n_kv, S_out]
  int* kept;              // [B, n_kv, budget]
  int* new_len;           // [B], may be kv_len
  int* old_len;           // [B] scratch: kv_len as the selection read it (-1: out of range)
  int* status;
};

// Rotation of heads by position (attn_rope_apply), or the table of it.
struct RopeParams {
  gqa_rope rope;
  int n_tok, n_heads;
  int heads_each;          // heads that one warp takes of a token (of 4 at a time)
  long long stride, out_stride;
  const void* x;           // bf16
  const int* positions;    // [n_tok]
  void* out;               // bf16, may be x; table: fp32 [n_tok, 64, 2]
};

// A pool of cache pages: element d of head g in slot i of page n is at n page + i pos + g head + d.
struct PagedPool {
  int n_pages, page_size;
  long long page, pos, head;  // elements
  void* k;
  void* v;
  const float* k_scale;    // [n_kv] of e4m3 pools, or null
  const float* v_scale;
};

struct PagedAppendParams {
  gqa_rope rope;
  int rotate;              // 0: keys as they are
  int B, T, n_kv, max_pages;
  long long stride_b, stride_t;
  PagedPool pool;
  const void* k;
  const void* v;
  const int* rope_pos;     // [B] or null: kv_len
  const int* page_table;   // [B, max_pages]
  const int* kv_len;       // [B]
  const int* n_new;        // [B] or null: T
  int* status;
};

// Attention of one token per sequence over pages: keys 0 .. kv_len[b] + n_new - 1.
struct PagedAttnParams {
  int B, n_kv, n_new, max_pages;
  PagedPool pool;
  const void* q;           // [B, 512 n_kv] bf16
  const int* page_table;   // [B, max_pages]
  const int* kv_len;       // [B]
  void* h;                 // [B, 512 n_kv] bf16
  int S_max;               // max_pages x page_size
  int log_box;             // slots of a copy, a power of two that divides the page
  int unit_cost;           // empty places of a unit in the CTAs' shares (kv_sched.h)
  float* part_o;           // partial results of cut units: [2 CTAs][4 heads][128]
  float2* part_ml;         // their (maximum, sum): [2 CTAs][4]
  int* counters;           // [B n_kv] pieces of a unit that have arrived (zero between calls)
  int* group_counters;     // [2 CTAs] the same of a group of a unit's pieces
  int* status;
  int fault;               // test hook: the last worker issues no loads (its waits run out)
  float scale_log2;        // log2(e) / sqrt(128)
};

}  // namespace gqa
