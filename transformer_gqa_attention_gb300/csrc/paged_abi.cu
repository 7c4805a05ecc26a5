// paged_abi.cu — the entry points of include/gqa_attn.h for paged caches and rotations: the set-up of
// a rotation, its application, the description of a paged cache, the append to it and the attention
// over it.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>

#include "ctx.h"
#include "gqa_attn.h"
#include "kv_sched.h"
#include "launch.h"
#include "paged_call.h"
#include "params.h"

using namespace gqa;

namespace {

constexpr int kRopeCheck = 0x726f7065;

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

bool valid(const gqa_rope* r) {
  return r->check == kRopeCheck && (r->layout == GQA_ROPE_PAIRS || r->layout == GQA_ROPE_HALVES) && r->rot_dim >= 16 &&
         r->rot_dim <= 128 && r->rot_dim % 16 == 0;
}

// w of pair j, scaled.
double frequency(int rot_dim, int j, double theta, const gqa_rope_scaling& s) {
  constexpr double kTwoPi = 6.283185307179586476925;
  const double w = std::pow(theta, -2.0 * j / rot_dim);
  switch (s.kind) {
    case GQA_ROPE_LINEAR: return w / s.factor;
    case GQA_ROPE_BANDS: {
      const double turns = s.context * w / kTwoPi;  // over the original context
      if (turns > s.high) return w;
      if (turns < s.low) return w / s.factor;
      const double m = (turns - s.low) / (s.high - s.low);
      return (1.0 - m) * w / s.factor + m * w;
    }
    case GQA_ROPE_RAMP: {
      auto pair = [&](double n) { return rot_dim * std::log(s.context / (n * kTwoPi)) / (2.0 * std::log(theta)); };
      const double a = std::max(std::floor(pair(s.high)), 0.0);
      const double b = std::min(std::ceil(pair(s.low)), rot_dim - 1.0);
      const double m = std::min(std::max((j - a) / std::max(b - a, 0.001), 0.0), 1.0);
      return m * w / s.factor + (1.0 - m) * w;
    }
    default: return w;
  }
}

// Elements from a row's start that rows 0 .. n - 1 of `stride` reach.
size_t reach(long long n, long long stride) { return static_cast<size_t>(n - 1) * static_cast<size_t>(stride); }

long long floor_div(long long x, long long y) { return x / y - (x % y < 0); }

// Whether rows of `row` bytes of two pools with these extents (the narrowest first) meet, the second one's `d` bytes
// behind the first one's: of each extent no more than two steps bring them within reach of one another.
bool rows_meet(const PagedExtent* e, int dims, long long row, long long d) {
  if (dims == 0) return d > -row && d < row;
  const PagedExtent& w = e[dims - 1];
  const long long first = std::max(floor_div(-w.below - d, w.stride) + 1, 1 - w.n);
  const long long last = std::min(-floor_div(d - w.below, w.stride) - 1, w.n - 1);
  for (long long k = first; k <= last; ++k)
    if (rows_meet(e, dims - 1, row, d + k * w.stride)) return true;
  return false;
}

// Whether bytes lo .. hi - 1 from a pool's start on hold some of a row: of three steps of an extent that they touch, the
// middle one lies whole within them.
bool rows_touch(const PagedExtent* e, int dims, long long row, long long lo, long long hi) {
  if (dims == 0) return lo < row && hi > 0;
  const PagedExtent& w = e[dims - 1];
  const long long first = std::max(floor_div(lo - w.below, w.stride) + 1, 0LL);
  const long long last = std::min(-floor_div(-hi, w.stride) - 1, w.n - 1);
  if (last - first >= 2) return true;
  for (long long i = first; i <= last; ++i)
    if (rows_touch(e, dims - 1, row, lo - i * w.stride, hi - i * w.stride)) return true;
  return false;
}
// Whether `bytes` at p hold some of what a description's calls read: rows of either pool, or scales.
bool holds_some(const gqa_paged* g, const void* p, size_t bytes) {
  const long long row = g->dtype == GQA_CACHE_BF16 ? 256 : 128;
  for (const void* pool : {g->pool.k, g->pool.v}) {
    const long long lo = static_cast<long long>(reinterpret_cast<intptr_t>(p) - reinterpret_cast<intptr_t>(pool));
    if (rows_touch(g->extents, g->n_extents, row, lo, lo + static_cast<long long>(bytes))) return true;
  }
  for (const float* scales : {g->pool.k_scale, g->pool.v_scale})
    if (scales && overlap(p, bytes, scales, 4 * static_cast<size_t>(g->n_kv))) return true;
  return false;
}

// A pool as the attention copies it: boxes of 2^log_box slots of one head and page, bf16 rows as two halves of
// 64 elements.
bool map_pool(CUtensorMap* m, const void* base, const gqa_paged* g) {
  const PagedPool& p = g->pool;
  const uint64_t n_pages = p.n_pages, slots = p.page_size, heads = g->n_kv;
  const uint32_t box = 1u << g->log_box;
  if (g->dtype == GQA_CACHE_E4M3) {
    const uint64_t dims[4] = {128, slots, heads, n_pages};
    const uint64_t strides[3] = {static_cast<uint64_t>(p.pos), static_cast<uint64_t>(p.head), static_cast<uint64_t>(p.page)};
    const uint32_t shape[4] = {128, box, 1, 1};
    return make_map(m, base, 4, dims, strides, shape, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
  }
  const uint64_t dims[5] = {64, slots, 2, heads, n_pages};
  const uint64_t strides[4] = {2 * static_cast<uint64_t>(p.pos), 128, 2 * static_cast<uint64_t>(p.head),
                               2 * static_cast<uint64_t>(p.page)};
  const uint32_t shape[5] = {64, box, 2, 1, 1};
  return make_map(m, base, 5, dims, strides, shape);
}

// Scratch of the attention: partial results of at most two pieces a CTA.
struct PagedScratch {
  int ctas;
  size_t part_o, part_ml, bytes;
};
PagedScratch paged_scratch(const gqa_ctx* c) {
  PagedScratch l{};
  l.ctas = std::min(2 * c->num_sms, kGroupCounterInts / 2);
  const size_t rows = 2 * static_cast<size_t>(l.ctas) * 4;
  l.part_ml = round_up(rows * 128 * sizeof(float), 256);
  l.bytes = l.part_ml + rows * sizeof(float2);
  return l;
}

size_t pool_bytes(const gqa_paged* g) {
  const PagedPool& p = g->pool;
  return (reach(p.n_pages, p.page) + reach(p.page_size, p.pos) + reach(g->n_kv, p.head) + 128) *
         (g->dtype == GQA_CACHE_BF16 ? 2 : 1);
}

}  // namespace

gqa_status gqa::check_paged(gqa_ctx* c, const gqa_paged* g, int max_pages) {
  if (g->n_kv != c->n_kv) return GQA_ERR_INVALID_ARG;
  if (g->device != c->device) return GQA_ERR_DEVICE;
  if (static_cast<long long>(max_pages) * g->pool.page_size > kMaxSMax) return GQA_ERR_SHAPE;
  return GQA_OK;
}

gqa_status gqa::reserve_paged_attn(gqa_ctx* c, cudaStream_t s) {
  return ensure_buffer(c, c->cache_ws, paged_scratch(c).bytes, s);
}

gqa_status gqa::run_paged_append(gqa_ctx* c, const gqa_paged* g, const PagedAppendCall& a, cudaStream_t s) {
  PagedAppendParams p{};
  if (a.rope) p.rope = *a.rope;
  p.rotate = a.rope != nullptr;
  p.B = a.B;
  p.T = a.T;
  p.n_kv = c->n_kv;
  p.max_pages = a.max_pages;
  p.stride_b = a.stride_b;
  p.stride_t = a.stride_t;
  p.pool = g->pool;
  p.k = a.k;
  p.v = a.v;
  p.rope_pos = a.rope_pos;
  p.page_table = a.page_table;
  p.kv_len = a.kv_len;
  p.n_new = a.n_new;
  p.status = c->status;
  ProfScope ps(c, GQA_KERNEL_PAGED_APPEND, s);
  GQA_CUDA(launch_paged_append(p, g->dtype, s));
  return GQA_OK;
}

gqa_status gqa::run_paged_attn(gqa_ctx* c, const gqa_paged* g, const void* q, int B, const int* page_table,
                               int max_pages, const int* kv_len, int n_new, void* h, cudaStream_t s) {
  const PagedScratch l = paged_scratch(c);
  gqa_status st = ensure_buffer(c, c->cache_ws, l.bytes, s);
  if (st != GQA_OK) return st;
  PagedAttnParams p{};
  p.B = B;
  p.n_kv = c->n_kv;
  p.n_new = n_new;
  p.max_pages = max_pages;
  p.pool = g->pool;
  p.q = q;
  p.page_table = page_table;
  p.kv_len = kv_len;
  p.h = h;
  p.S_max = max_pages * g->pool.page_size;
  p.log_box = g->log_box;
  // (with 0, 1, 2 and 4, us: 16 sequences of up to 4096 keys 29.4, 28.4, 27.5, 27.6; 64 of up to 8192 e4m3 97, 92, 89, 90)
  p.unit_cost = kUnitCostDecode;
  p.part_o = reinterpret_cast<float*>(c->cache_ws.p + l.part_o);
  p.part_ml = reinterpret_cast<float2*>(c->cache_ws.p + l.part_ml);
  p.counters = c->counters;
  p.group_counters = c->counters + kCounterInts;
  p.status = c->status;
  p.scale_log2 = kScaleLog2;
  p.fault = take_fault(c, GQA_KERNEL_PAGED_ATTN);
  // A CTA per range and kv head: as many as fit, or as the longest sequences that the table allows have places for (the host
  // does not know the lengths).  Under a table much wider than they need, for 131072 positions, one sequence of 700 keys
  // takes 5.9 us instead of 5.6 (e4m3 6.2 instead of 5.9: the kernel for many pieces, below, and CTAs without a range); 8 of
  // 300, 16 of up to 4000 and one of 131000 take the same.
  const size_t tiles = (static_cast<size_t>(p.S_max) + kKvTile - 1) / kKvTile;
  const int ranges = static_cast<int>(std::min<size_t>(l.ctas / c->n_kv, static_cast<size_t>(B) * (tiles + p.unit_cost)));
  // More than 16 pieces to a sequence if the lengths are alike and fill the table: joined in groups (one kv head, 32000 and 131000 keys: 19.4 -> 9.1
  // and 31.3 -> 18.7 us; 8 kv heads, 38 pieces each, 12000 keys 15.1 -> 14.5).  The others have a kernel of their own: with the
  // groups in it calls with a few pieces take 0.2 to 0.3 us more (of 5.8 to 25).  Either is right for any lengths.
  const bool groups = ranges > 16 * B;
  ProfScope ps(c, GQA_KERNEL_PAGED_ATTN, s);
  GQA_CUDA(launch_paged_attn(g->map_k, g->map_v, p, g->dtype, ranges * c->n_kv, groups, s));
  return GQA_OK;
}

extern "C" {

gqa_status attn_rope_init(gqa_rope* rope, int layout, int rot_dim, double theta, const gqa_rope_scaling* scaling) {
  if (!rope || (layout != GQA_ROPE_PAIRS && layout != GQA_ROPE_HALVES)) return GQA_ERR_INVALID_ARG;
  if (rot_dim < 16 || rot_dim > 128 || rot_dim % 16) return GQA_ERR_SHAPE;
  gqa_rope_scaling s{};
  if (scaling) s = *scaling;
  if (!std::isfinite(theta) || !(theta > 1.0) || s.kind < GQA_ROPE_PLAIN || s.kind > GQA_ROPE_RAMP) return GQA_ERR_INVALID_ARG;
  if (s.kind != GQA_ROPE_PLAIN && (!std::isfinite(s.factor) || !(s.factor >= 1.0))) return GQA_ERR_INVALID_ARG;
  if ((s.kind == GQA_ROPE_BANDS || s.kind == GQA_ROPE_RAMP) &&
      (!std::isfinite(s.context) || !(s.context > 0.0) || !(s.low > 0.0) || !std::isfinite(s.high) || !(s.high > s.low)))
    return GQA_ERR_INVALID_ARG;
  *rope = gqa_rope{};
  for (int j = 0; j < rot_dim / 2; ++j)  // w <= 1: less than a sixth of a revolution
    rope->turns[j] =
        static_cast<unsigned long long>(frequency(rot_dim, j, theta, s) * (18446744073709551616.0 / 6.283185307179586476925));
  rope->gain = s.kind == GQA_ROPE_RAMP ? static_cast<float>(0.1 * std::log(s.factor) + 1.0) : 1.f;
  rope->layout = layout;
  rope->rot_dim = rot_dim;
  rope->check = kRopeCheck;
  return GQA_OK;
}

gqa_status attn_rope_apply(gqa_ctx* c, const gqa_rope* rope, const void* x, int n_tok, int n_heads, long long stride,
                           const int* positions, void* out, long long out_stride, gqa_stream_t stream) {
  if (!c || !rope || !x || !positions || !out || !valid(rope)) return GQA_ERR_INVALID_ARG;
  const long long width = 128LL * n_heads, most = 1LL << 31;
  if (n_tok < 1 || n_tok > kMaxTokens || n_heads < 1 || n_heads > 1024 || stride < width || out_stride < width ||
      stride >= most || out_stride >= most)
    return GQA_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(positions) || !aligned16(out) || stride % 8 || out_stride % 8) return GQA_ERR_ALIGN;
  const size_t in_bytes = 2 * (reach(n_tok, stride) + width), out_bytes = 2 * (reach(n_tok, out_stride) + width);
  if (!(out == x && (out_stride == stride || n_tok == 1)) && overlap(out, out_bytes, x, in_bytes)) return GQA_ERR_INVALID_ARG;
  if (overlap(out, out_bytes, positions, 4 * static_cast<size_t>(n_tok))) return GQA_ERR_INVALID_ARG;
  gqa_status st = check_device(c);
  if (st != GQA_OK) return st;
  CallRange range("gqa.attn_rope_apply");
  RopeParams p{};
  p.rope = *rope;
  p.n_tok = n_tok;
  p.n_heads = n_heads;
  p.heads_each = n_heads;
  p.stride = stride;
  p.out_stride = out_stride;
  p.x = x;
  p.positions = positions;
  p.out = out;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  ProfScope ps(c, GQA_KERNEL_ROPE, s);
  GQA_CUDA(launch_rope_apply(p, s));
  return GQA_OK;
}

gqa_status attn_rope_table(gqa_ctx* c, const gqa_rope* rope, const int* positions, int n_tok, float* R,
                           gqa_stream_t stream) {
  if (!c || !rope || !positions || !R || !valid(rope) || rope->layout != GQA_ROPE_PAIRS) return GQA_ERR_INVALID_ARG;
  if (n_tok < 1 || n_tok > kMaxTokens) return GQA_ERR_SHAPE;
  if (!aligned16(positions) || !aligned16(R)) return GQA_ERR_ALIGN;
  if (overlap(R, 512 * static_cast<size_t>(n_tok), positions, 4 * static_cast<size_t>(n_tok))) return GQA_ERR_INVALID_ARG;
  gqa_status st = check_device(c);
  if (st != GQA_OK) return st;
  CallRange range("gqa.attn_rope_table");
  RopeParams p{};
  p.rope = *rope;
  p.n_tok = n_tok;
  p.positions = positions;
  p.out = R;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  ProfScope ps(c, GQA_KERNEL_ROPE, s);
  GQA_CUDA(launch_rope_table(p, s));
  return GQA_OK;
}

gqa_status attn_paged_create(gqa_ctx* c, void* k_pages, void* v_pages, int n_pages, int page_size, int dtype,
                             long long stride_page, long long stride_pos, long long stride_head, const float* k_scale,
                             const float* v_scale, gqa_paged** out) {
  if (!out) return GQA_ERR_INVALID_ARG;
  *out = nullptr;
  if (!c || !k_pages || !v_pages || k_pages == v_pages || (dtype != GQA_CACHE_BF16 && dtype != GQA_CACHE_E4M3) ||
      (dtype == GQA_CACHE_BF16 && (k_scale || v_scale)))
    return GQA_ERR_INVALID_ARG;
  if (n_pages < 1 || page_size < 8 || page_size % 8 || page_size > kMaxSMax) return GQA_ERR_SHAPE;
  if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k_scale) || !aligned16(v_scale)) return GQA_ERR_ALIGN;
  const int size = dtype == GQA_CACHE_BF16 ? 2 : 1;
  // dimensions with more than one entry, the narrowest stride first: each has to step over all of those before
  PagedExtent dims[3]{};
  int used = 0;
  const PagedExtent all[3] = {{n_pages, stride_page, 0}, {page_size, stride_pos, 0}, {c->n_kv, stride_head, 0}};
  for (const PagedExtent& d : all)
    if (d.n > 1) {
      if (d.stride < 1 || d.stride >= (1LL << 39) / size || d.stride > (1LL << 46) / d.n) return GQA_ERR_SHAPE;
      if (d.stride * size % 16) return GQA_ERR_ALIGN;
      dims[used++] = {d.n, d.stride * size, 0};
    }
  std::sort(dims, dims + used, [](const PagedExtent& a, const PagedExtent& b) { return a.stride < b.stride; });
  long long reached = 128 * size;
  for (int i = 0; i < used; ++i) {
    if (dims[i].stride < reached) return GQA_ERR_INVALID_ARG;
    dims[i].below = reached;
    reached += dims[i].stride * (dims[i].n - 1);
  }
  if (rows_meet(dims, used, 128 * size, static_cast<long long>(reinterpret_cast<intptr_t>(v_pages) - reinterpret_cast<intptr_t>(k_pages))))
    return GQA_ERR_INVALID_ARG;
  gqa_paged* g = new (std::nothrow) gqa_paged();
  if (!g) return GQA_ERR_OOM;
  g->device = c->device;
  g->n_kv = c->n_kv;
  g->dtype = dtype;
  g->pool = {n_pages,
             page_size,
             n_pages > 1 ? stride_page : 128,
             stride_pos,
             c->n_kv > 1 ? stride_head : 128,
             k_pages,
             v_pages,
             k_scale,
             v_scale};
  g->n_extents = used;
  std::copy(dims, dims + 3, g->extents);
  for (g->log_box = 3; g->log_box < 6 && page_size % (2 << g->log_box) == 0;) ++g->log_box;
  if (!map_pool(&g->map_k, k_pages, g) || !map_pool(&g->map_v, v_pages, g)) {
    delete g;
    return cuda_fail(cudaErrorInvalidValue);
  }
  *out = g;
  return GQA_OK;
}

void attn_paged_destroy(gqa_paged* g) { delete g; }

gqa_status attn_paged_append(gqa_ctx* c, const gqa_paged* g, const void* k, const void* v, int B, int T,
                             long long stride_b, long long stride_t, const gqa_rope* rope, const int* rope_pos,
                             const int* page_table, int max_pages, const int* kv_len, const int* n_new,
                             gqa_stream_t stream) {
  if (!c || !g || !k || !v || !page_table || !kv_len || (rope && !valid(rope))) return GQA_ERR_INVALID_ARG;
  if (B < 1 || B > kDecodeMaxBatch || T < 1 || static_cast<long long>(B) * T > kMaxTokens || max_pages < 1) return GQA_ERR_SHAPE;
  if (!aligned16(k) || !aligned16(v) || !aligned16(rope_pos) || !aligned16(page_table) || !aligned16(kv_len) ||
      !aligned16(n_new))
    return GQA_ERR_ALIGN;
  if (B == 1) stride_b = 0;
  if (T == 1) stride_t = 0;
  if (stride_b % 8 || stride_t % 8) return GQA_ERR_ALIGN;
  if (stride_b < 0 || stride_t < 0 || stride_b >= 1LL << 31 || stride_t >= 1LL << 31) return GQA_ERR_SHAPE;
  gqa_status st = check_device(c);
  if (st != GQA_OK) return st;
  if ((st = check_paged(c, g, max_pages)) != GQA_OK) return st;
  const long long width = 128LL * c->n_kv;
  if ((T > 1 && stride_t < width) || (B > 1 && stride_b < width)) return GQA_ERR_SHAPE;
  const size_t rows = 2 * (reach(B, stride_b) + reach(T, stride_t) + width), pool = pool_bytes(g);
  for (const void* src : {k, v})
    for (const void* dst : {g->pool.k, g->pool.v})
      if (overlap(src, rows, dst, pool)) return GQA_ERR_INVALID_ARG;
  CallRange range("gqa.attn_paged_append");
  PagedAppendCall a{};
  a.k = k;
  a.v = v;
  a.B = B;
  a.T = T;
  a.stride_b = stride_b;
  a.stride_t = stride_t;
  a.rope = rope;
  a.rope_pos = rope_pos;
  a.page_table = page_table;
  a.max_pages = max_pages;
  a.kv_len = kv_len;
  a.n_new = n_new;
  return run_paged_append(c, g, a, reinterpret_cast<cudaStream_t>(stream));
}

gqa_status attn_paged_decode_attention(gqa_ctx* c, const gqa_paged* g, const void* q_r, int B, const int* page_table,
                                       int max_pages, const int* kv_len, void* h, gqa_stream_t stream) {
  if (!c || !g || !q_r || !page_table || !kv_len || !h) return GQA_ERR_INVALID_ARG;
  if (B < 1 || B > kDecodeMaxBatch || max_pages < 1) return GQA_ERR_SHAPE;
  if (!aligned16(q_r) || !aligned16(page_table) || !aligned16(kv_len) || !aligned16(h)) return GQA_ERR_ALIGN;
  gqa_status st = check_device(c);
  if (st != GQA_OK) return st;
  if ((st = check_paged(c, g, max_pages)) != GQA_OK) return st;
  const size_t heads = static_cast<size_t>(B) * c->n_kv * 1024;
  if (overlap(h, heads, q_r, heads) || overlap(h, heads, kv_len, 4 * static_cast<size_t>(B)) ||
      overlap(h, heads, page_table, 4 * static_cast<size_t>(B) * max_pages) || holds_some(g, h, heads))
    return GQA_ERR_INVALID_ARG;
  CallRange range("gqa.attn_paged_decode_attention");
  return run_paged_attn(c, g, q_r, B, page_table, max_pages, kv_len, 0, h, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
