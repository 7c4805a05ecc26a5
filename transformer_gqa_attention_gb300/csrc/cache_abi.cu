// cache_abi.cu — the entry points of include/gqa_attn.h that work on a cache directly: tree
// attention, decode attention with accumulated key weights, commit of an accepted path and
// eviction by weight.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "cache_call.h"
#include "ctx.h"
#include "gqa_attn.h"
#include "kv_sched.h"
#include "launch.h"
#include "params.h"

using namespace gqa;

namespace {

// What a call keeps in the context's scratch, in bytes from its start.
struct CacheLayout {
  bool pair;
  int group_pos, row_groups, unit_cost, part_rows, n_ctas;
  size_t tiles, workers;  // tiles: at most
  size_t merge, part_ml, part_o, total_tiles, scores, tile_unit, unit_ml, bytes;
};

CacheLayout cache_layout(const gqa_ctx* c, const CacheAttnCall& a) {
  CacheLayout l{};
  l.pair = a.T > kOneTilePos;
  l.group_pos = l.pair ? 64 : kOneTilePos;
  l.row_groups = (a.T + l.group_pos - 1) / l.group_pos;
  l.unit_cost = a.weights ? kUnitCostDecode : l.pair ? kUnitCostPair : kUnitCostTile;
  l.part_rows = static_cast<int>(round_up(4 * std::min(a.T, l.group_pos), 32));
  auto take = [&](size_t bytes) {
    const size_t at = l.bytes;
    l.bytes = round_up(l.bytes + bytes, 256);
    return at;
  };
  // persistent CTAs, one per SM (the GPU's 152: even), or as many as the caches have places for
  const size_t units = static_cast<size_t>(a.B) * c->n_kv * l.row_groups;
  l.tiles = units * ((a.S_max + kKvTile - 1) / kKvTile);
  const size_t places = l.tiles + units * l.unit_cost, ctas = c->num_sms & ~1;
  l.n_ctas = static_cast<int>(std::min(ctas, a.weights ? (places + 1) / 2 : l.pair ? 2 * places : places));
  // workers: CTAs, with weights their two softmax slots, with many positions CTA pairs; each may hold
  // two partial results
  l.workers = a.weights ? 2 * l.n_ctas : l.pair ? l.n_ctas / 2 : l.n_ctas;
  const size_t slots = 2 * l.workers;
  l.merge = take(l.workers * sizeof(int4));
  l.part_ml = take(slots * l.part_rows * sizeof(float2));
  l.part_o = take(slots * l.part_rows * 128 * sizeof(float));
  if (a.weights) {
    l.total_tiles = take(sizeof(int));
    l.scores = take(l.tiles * 4 * kKvTile * sizeof(float));
    l.tile_unit = take(l.tiles * sizeof(int4));
    l.unit_ml = take(units * 4 * sizeof(float2));
  }
  return l;
}

}  // namespace

gqa_status gqa::reserve_cache_attn(gqa_ctx* c, const CacheAttnCall& a, cudaStream_t s) {
  return ensure_buffer(c, c->cache_ws, cache_layout(c, a).bytes, s);
}

gqa_status gqa::run_cache_attn(gqa_ctx* c, const CacheAttnCall& a, cudaStream_t s) {
  const int G = c->n_kv;
  const CacheLayout l = cache_layout(c, a);
  gqa_status st = ensure_buffer(c, c->cache_ws, l.bytes, s);
  if (st != GQA_OK) return st;
  uint8_t* ws = c->cache_ws.p;
  CacheAttnParams p{};
  p.B = a.B;
  p.T = a.T;
  p.S_max = a.S_max;
  p.n_kv = G;
  p.n_new = a.n_new;
  p.mask = a.mask;
  p.kv_len = a.kv_len;
  p.h = a.h;
  p.weights = a.weights;
  p.status = c->status;
  p.scale_log2 = kScaleLog2;
  p.group_pos = l.group_pos;
  p.row_groups = l.row_groups;
  p.unit_cost = l.unit_cost;
  p.part_rows = l.part_rows;
  p.merge = reinterpret_cast<int4*>(ws + l.merge);
  p.part_ml = reinterpret_cast<float2*>(ws + l.part_ml);
  p.part_o = reinterpret_cast<float*>(ws + l.part_o);
  if (a.weights) {
    p.total_tiles = reinterpret_cast<int*>(ws + l.total_tiles);
    p.scores = reinterpret_cast<float*>(ws + l.scores);
    p.tile_unit = reinterpret_cast<int4*>(ws + l.tile_unit);
    p.unit_ml = reinterpret_cast<float2*>(ws + l.unit_ml);
  }

  CUtensorMap tq, tk, tv;
  // queries as (d, head, position, sequence): a box is 64 d of the group's 4 heads
  const uint64_t dims[4] = {128, 4ull * G, static_cast<uint64_t>(a.T), static_cast<uint64_t>(a.B)};
  const uint64_t strides[3] = {256, static_cast<uint64_t>(G) * 1024, static_cast<uint64_t>(a.T) * G * 1024};
  const uint32_t box[4] = {64, 4, a.weights ? 1u : kOneTilePos, 1};
  if (!make_map(&tq, a.q, 4, dims, strides, box) ||
      !map_cache(&tk, a.cache_k, a.B, a.S_max, G, a.S_max, l.pair ? kKvTile / 2 : kKvTile) ||
      !map_cache(&tv, a.cache_v, a.B, a.S_max, G, a.S_max, kKvTile))
    return cuda_fail(cudaErrorInvalidValue);
  p.fault = take_fault(c, GQA_KERNEL_CACHE_ATTN);
  {
    ProfScope ps(c, GQA_KERNEL_CACHE_ATTN, s);
    GQA_CUDA(launch_cache_attn(tq, tk, tv, p, l.n_ctas, s));
  }
  if (a.weights) {
    ProfScope ps(c, GQA_KERNEL_CACHE_WEIGHTS, s);
    // a warp per tile, at most four blocks per SM (two: 7 us more for 64 sequences of 8192 keys; eight: 1 us more
    // for one of 700)
    const int blocks = static_cast<int>(std::min<size_t>(4 * c->num_sms, (l.tiles + 7) / 8));
    GQA_CUDA(launch_cache_weights(p, static_cast<int>(l.workers), blocks, s));
  } else {
    ProfScope ps(c, GQA_KERNEL_CACHE_MERGE, s);
    GQA_CUDA(launch_cache_merge(p, static_cast<int>(l.workers), s));
  }
  return GQA_OK;
}

namespace {

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

}  // namespace

extern "C" {

gqa_status attn_tree_attention(gqa_ctx* c, const void* q_r, int B, int T, const unsigned* tree_mask,
                               const void* cache_k, const void* cache_v, int S_max, const int* prefix_len, void* h,
                               gqa_stream_t stream) {
  if (!c || !q_r || !tree_mask || !cache_k || !cache_v || !prefix_len || !h) return GQA_ERR_INVALID_ARG;
  if (B < 1 || B > kDecodeMaxBatch || T < 1 || T > GQA_MAX_TREE || S_max < 1 || S_max > kMaxSMax || T > S_max)
    return GQA_ERR_SHAPE;
  if (!aligned16(q_r) || !aligned16(tree_mask) || !aligned16(cache_k) || !aligned16(cache_v) ||
      !aligned16(prefix_len) || !aligned16(h))
    return GQA_ERR_ALIGN;
  gqa_status st = check_device(c);
  if (st != GQA_OK) return st;
  CallRange range("gqa.attn_tree_attention");
  CacheAttnCall a{};
  a.B = B;
  a.T = T;
  a.n_new = T;
  a.S_max = S_max;
  a.mask = tree_mask;
  a.kv_len = prefix_len;
  a.q = q_r;
  a.cache_k = cache_k;
  a.cache_v = cache_v;
  a.h = h;
  return run_cache_attn(c, a, reinterpret_cast<cudaStream_t>(stream));
}

gqa_status attn_decode_attention_weights(gqa_ctx* c, const void* q_r, const void* cache_k, const void* cache_v, int B,
                                         int S_max, const int* kv_len, float* weights, void* h,
                                         gqa_stream_t stream) {
  if (!c || !q_r || !cache_k || !cache_v || !kv_len || !weights || !h) return GQA_ERR_INVALID_ARG;
  if (B < 1 || B > kDecodeMaxBatch || S_max < 1 || S_max > kMaxSMax) return GQA_ERR_SHAPE;
  if (!aligned16(q_r) || !aligned16(cache_k) || !aligned16(cache_v) || !aligned16(kv_len) || !aligned16(weights) ||
      !aligned16(h))
    return GQA_ERR_ALIGN;
  gqa_status st = check_device(c);
  if (st != GQA_OK) return st;
  CallRange range("gqa.attn_decode_attention_weights");
  CacheAttnCall a{};
  a.B = B;
  a.T = 1;
  a.n_new = 0;
  a.S_max = S_max;
  a.kv_len = kv_len;
  a.q = q_r;
  a.cache_k = cache_k;
  a.cache_v = cache_v;
  a.h = h;
  a.weights = weights;
  return run_cache_attn(c, a, reinterpret_cast<cudaStream_t>(stream));
}

gqa_status attn_cache_commit(gqa_ctx* c, void* cache_k, void* cache_v, int B, int S_max, int T, const int* prefix_len,
                             const int* path, const int* n_accept, int* new_len, gqa_stream_t stream) {
  if (!c || !cache_k || !cache_v || !prefix_len || !path || !n_accept || !new_len) return GQA_ERR_INVALID_ARG;
  if (B < 1 || B > kDecodeMaxBatch || T < 1 || T > GQA_MAX_TREE || S_max < 1 || S_max > kMaxSMax || T > S_max)
    return GQA_ERR_SHAPE;
  if (!aligned16(cache_k) || !aligned16(cache_v) || !aligned16(prefix_len) || !aligned16(path) ||
      !aligned16(n_accept) || !aligned16(new_len))
    return GQA_ERR_ALIGN;
  const size_t lens = static_cast<size_t>(B) * sizeof(int);
  if ((new_len != prefix_len && overlap(new_len, lens, prefix_len, lens)) || overlap(new_len, lens, n_accept, lens) ||
      overlap(new_len, lens, path, lens * T))
    return GQA_ERR_INVALID_ARG;
  gqa_status st = check_device(c);
  if (st != GQA_OK) return st;
  const size_t bytes = static_cast<size_t>(B) * S_max * c->n_kv * 256;
  if (overlap(cache_k, bytes, cache_v, bytes)) return GQA_ERR_INVALID_ARG;
  CallRange range("gqa.attn_cache_commit");
  CommitParams p{};
  p.B = B;
  p.S_max = S_max;
  p.T = T;
  p.n_kv = c->n_kv;
  p.k = cache_k;
  p.v = cache_v;
  p.prefix_len = prefix_len;
  p.path = path;
  p.n_accept = n_accept;
  p.new_len = new_len;
  p.status = c->status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  ProfScope ps(c, GQA_KERNEL_CACHE_COMMIT, s);
  GQA_CUDA(launch_cache_commit(p, s));
  return GQA_OK;
}

gqa_status attn_cache_evict(gqa_ctx* c, const void* cache_k, const void* cache_v, const float* weights, int B,
                            int S_max, const int* kv_len, int budget, int n_first, int n_recent, void* out_k,
                            void* out_v, float* out_weights, int S_out, int* kept, int* new_len,
                            gqa_stream_t stream) {
  if (!c || !cache_k || !cache_v || !weights || !kv_len || !out_k || !out_v || !out_weights || !kept || !new_len)
    return GQA_ERR_INVALID_ARG;
  if (B < 1 || B > kDecodeMaxBatch || S_max < 1 || S_max > kMaxSMax || S_out < 1 || S_out > kMaxSMax || budget < 1 ||
      budget > S_out || n_first < 0 || n_recent < 0 || static_cast<long long>(n_first) + n_recent > budget)
    return GQA_ERR_SHAPE;
  if (!aligned16(cache_k) || !aligned16(cache_v) || !aligned16(weights) || !aligned16(kv_len) || !aligned16(out_k) ||
      !aligned16(out_v) || !aligned16(out_weights) || !aligned16(kept) || !aligned16(new_len))
    return GQA_ERR_ALIGN;
  // either every output is its input (in place) or none overlaps any of them
  const bool in_place = out_k == cache_k && out_v == cache_v && out_weights == weights && S_out == S_max;
  const void* ins[3] = {cache_k, cache_v, weights};
  const void* outs[3] = {out_k, out_v, out_weights};
  for (int i = 0; i < 3 && !in_place; ++i)
    for (int j = 0; j < 3; ++j)
      if (ins[i] == outs[j]) return GQA_ERR_INVALID_ARG;
  const size_t lens = static_cast<size_t>(B) * sizeof(int);
  if (new_len != kv_len && overlap(new_len, lens, kv_len, lens)) return GQA_ERR_INVALID_ARG;
  gqa_status st = check_device(c);
  if (st != GQA_OK) return st;
  // no output overlaps another, nor an input other than its own (in place; new_len: kv_len)
  const size_t unit = static_cast<size_t>(B) * c->n_kv;  // (sequence, kv head) pairs; 256 bytes of K per position
  const size_t in_bytes[4] = {unit * S_max * 256, unit * S_max * 256, unit * S_max * 4, lens};
  const size_t out_bytes[5] = {unit * S_out * 256, unit * S_out * 256, unit * S_out * 4, lens, unit * budget * 4};
  const void* all_ins[4] = {cache_k, cache_v, weights, kv_len};
  const void* all_outs[5] = {out_k, out_v, out_weights, new_len, kept};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(all_outs[i], out_bytes[i], all_outs[j], out_bytes[j])) return GQA_ERR_INVALID_ARG;
    for (int j = 0; j < 4; ++j) {
      const bool own = i == j && all_outs[i] == all_ins[j] && (i == 3 || in_place);
      if (!own && overlap(all_outs[i], out_bytes[i], all_ins[j], in_bytes[j])) return GQA_ERR_INVALID_ARG;
    }
  }
  CallRange range("gqa.attn_cache_evict");
  EvictParams p{};
  p.B = B;
  p.S_max = S_max;
  p.S_out = S_out;
  p.n_kv = c->n_kv;
  p.budget = budget;
  p.n_first = n_first;
  p.n_recent = n_recent;
  p.in_place = in_place ? 1 : 0;
  p.k = cache_k;
  p.v = cache_v;
  p.weights = weights;
  p.kv_len = kv_len;
  p.out_k = out_k;
  p.out_v = out_v;
  p.out_weights = out_weights;
  p.kept = kept;
  p.new_len = new_len;
  p.old_len = c->old_len;
  p.status = c->status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  {
    ProfScope ps(c, GQA_KERNEL_EVICT_SELECT, s);
    GQA_CUDA(launch_evict_select(p, s));
  }
  {
    ProfScope ps(c, GQA_KERNEL_EVICT_MOVE, s);
    GQA_CUDA(launch_evict_move(p, s));
  }
  return GQA_OK;
}

gqa_status attn_debug_cache_schedule(const int* lens, int B, int n_new, int S_max, int units, int unit_cost, int workers,
                                     int* pieces, int max_pieces, int* n_pieces) {
  if (!lens || !n_pieces || (!pieces && max_pieces > 0) || B < 1 || n_new < 0 || S_max < 1 || units < 1 ||
      unit_cost < 0 || unit_cost > 64 || workers < 1 || workers > kMaxRangeWorkers || max_pieces < 0)
    return GQA_ERR_INVALID_ARG;
  auto len_of = [&](int b) { return b < B ? lens[b] : 0; };
  auto places_of = [&](int b) { return (kv_tiles(kv_end(len_of(b), n_new, S_max)) + unit_cost) * units; };
  long long all = 0;
  for (int b = 0; b < B; ++b) all += (static_cast<long long>(kv_tiles(kv_end(lens[b], n_new, S_max))) + unit_cost) * units;
  if (all > 0x7FFFFFFF) return GQA_ERR_SHAPE;
  const int total = static_cast<int>(all), n_work = range_workers(total, workers);
  int n = 0;
  for (int c = 0; c < n_work; ++c) {
    const int lo = range_start(total, n_work, c), hi = range_start(total, n_work, c + 1);
    int b = 0, at = 0;
    while (at + places_of(b) <= lo) at += places_of(b++);
    KvWalk w;
    for (w.start(unit_cost, b, lo - at, len_of(b), n_new, S_max, lo, hi - lo); !w.done(); w.next(units, n_new, S_max, len_of), ++n) {
      if (n < max_pieces) {
        int* o = pieces + 8 * n;
        o[0] = c;
        o[1] = w.b;
        o[2] = w.u;
        o[3] = w.first;
        o[4] = w.n;
        o[5] = w.whole() ? -1 : partial_slot(c, w.first > 0);
        o[6] = range_owner(total, n_work, w.place(w.tiles - 1));
        o[7] = w.tile(w.first, units);
      }
    }
  }
  *n_pieces = n;
  return n > max_pieces ? GQA_ERR_SHAPE : GQA_OK;
}

}  // extern "C"
