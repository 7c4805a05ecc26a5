/*
 * gqa_attn.h — C ABI of the GB300 (sm_103a) grouped-query attention block forward.
 *
 * The block is the Llama-3 / Llama-3.1 8B attention sub-block described on the page
 * "Llama 3.1 8B · Grouped-query attention" (step list "All 13 steps"; in/out contract
 * x [B,T,4096], R [T,64 pairs], M [T queries, T keys] -> Delta_attn [B,T,4096];
 * parameter table: W_Q 4096x4096, W_K and W_V 4096x(8x128), W_O 4096x4096).  It computes
 *
 *     Q = x W_Q,  K = x W_K,  V = x W_V                      (steps 1-3)
 *     Q_r, K_r = pair rotation of Q, K by R                  (steps 4-5)
 *     K_G[h] = K_r[h/4],  V_G[h] = V[h/4]                    (steps 6-7)
 *     S = Q_r K_G^T,  S_s = S / sqrt(128),  S_m = S_s + M    (steps 8-10)
 *     A = softmax over keys of S_m,  H = A V_G               (steps 11-12)
 *     H merged to [B,T,4096],  Delta_attn = H W_O            (steps 13-14)
 *
 * Dimensions are fixed by the model catalogue quoted on that page: dim 4096, 32 query
 * heads, 8 key/value heads, head width 128 (64 rotation pairs).  B, T, the cache length
 * S_max and start_pos are runtime values.
 *
 * Conventions shared by every call below
 *  - Every pointer argument named x, R, R_row, cache_k, cache_v, delta, wq, wk, wv, wo is
 *    a DEVICE pointer (cudaMalloc / torch CUDA storage on the current device).  The
 *    caller owns these buffers; the library borrows them for the duration of the
 *    asynchronous work it enqueues and never frees them.
 *  - bf16 tensors are IEEE bfloat16 bit patterns (uint16), row-major, densely packed.
 *  - Every device pointer must be 16-byte aligned (GQA_ERR_ALIGN otherwise).
 *  - `stream` is a cudaStream_t (NULL = legacy default stream).  All work is enqueued on
 *    it and the call returns without synchronising, except where noted.
 *  - Arguments are validated on the host before anything is enqueued; on any error the
 *    call enqueues nothing and returns a non-zero gqa_status.
 *  - A context may be used from one stream at a time; calls on one context must not
 *    overlap on different streams (they share the context's workspace).
 *  - Lengths that a call takes per sequence (prefix_len, kv_len, n_accept, path) are DEVICE
 *    int32 arrays, so a captured graph can be replayed with other lengths.  They are checked
 *    on the device: a sequence whose value is out of range is left out as the call says, the
 *    others are computed, and the next attn_sync_status returns GQA_ERR_SHAPE.
 *  - Memory that a call recorded into a CUDA graph uses stays allocated until attn_destroy,
 *    also when a later call needs a larger workspace.
 *  - Kernels bound every wait on the device.  A wait that runs out records
 *    GQA_ERR_TIMEOUT in the context's device status word and the kernel returns; read
 *    it with attn_sync_status.  Until it has been read, the outputs of later calls on the
 *    context are undefined as well.
 */
#ifndef GQA_ATTN_H
#define GQA_ATTN_H

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st; /* cudaStream_t is `struct CUstream_st *` */
typedef struct CUstream_st *gqa_stream_t;

typedef struct gqa_ctx gqa_ctx; /* opaque */

typedef enum {
    GQA_OK = 0,
    GQA_ERR_INVALID_ARG = 1, /* null pointer / null context / bad flag */
    GQA_ERR_SHAPE = 2,       /* B, T, S_max, start_pos (or a length read on the device) out of range */
    GQA_ERR_ALIGN = 3,       /* a device pointer is not 16-byte aligned */
    GQA_ERR_CUDA = 4,        /* a CUDA runtime call failed (see attn_last_cuda_error) */
    GQA_ERR_TIMEOUT = 5,     /* a bounded device-side wait ran out (device status word) */
    GQA_ERR_OOM = 6,         /* workspace allocation failed */
    GQA_ERR_DEVICE = 7       /* current device is not an sm_103 GPU */
} gqa_status;

#define GQA_DIM 4096
#define GQA_N_HEADS 32
#define GQA_N_KV_HEADS 8
#define GQA_HEAD_DIM 128
#define GQA_QKV_DIM 6144 /* 4096 query + 1024 key + 1024 value features */

/*
 * attn_create — build a context for one block on the current CUDA device.
 *
 * wq [4096,4096], wk [1024,4096], wv [1024,4096], wo [4096,4096]: bf16 device tensors in
 * the [out, in] storage of the quoted fairscale ColumnParallelLinear / RowParallelLinear
 * layers ("F.linear performs XA^T ... we allocate the transpose").  They are COPIED into
 * memory the context owns (W_Q, W_K, W_V packed into one [6144,4096] matrix; W_O kept
 * [4096,4096]); the caller may free its copies once the stream has passed this call.
 * The copies are enqueued on `stream`.
 * On success *out receives the context (to be released with attn_destroy).
 * Errors: GQA_ERR_INVALID_ARG (null), GQA_ERR_ALIGN, GQA_ERR_DEVICE (not sm_103),
 * GQA_ERR_OOM, GQA_ERR_CUDA.
 */
gqa_status attn_create(const void *wq, const void *wk, const void *wv, const void *wo,
                       gqa_stream_t stream, gqa_ctx **out);

/*
 * attn_create_shard — a context for one tensor-parallel shard of the block: the query heads
 * of n_kv_local consecutive kv groups (4 n_kv_local query heads, n_kv_local key/value
 * heads), as the quoted Attention.__init__ splits the block over model-parallel ranks
 * (page "Llama 3.1 8B · Grouped-query attention", Query projection: n_local_heads =
 * n_heads / model_parallel_size, n_local_kv_heads likewise; wq, wk, wv are
 * ColumnParallelLinear(gather_output=False), whose weight is [output_size_per_partition,
 * in_features]) and the output projection is a RowParallelLinear(input_is_parallel=True)
 * whose weight is [out_features, input_size_per_partition] (page "Llama 3.1 8B · Merge and
 * project").  Rank r of a world of w ranks holds kv groups 8r/w .. 8(r+1)/w - 1.
 *
 * wq_shard [512 n,4096]: rows 512 g0 .. 512 (g0+n) - 1 of W_Q (query heads 4 g0 .. 4 (g0+n) - 1)
 * wk_shard, wv_shard [128 n,4096]: rows 128 g0 .. 128 (g0+n) - 1 of W_K, W_V
 * wo_shard [4096,512 n]: columns 512 g0 .. 512 (g0+n) - 1 of W_O, row-major (densely packed)
 * with n = n_kv_local in 1..8; all bf16 device tensors, copied into the context as by
 * attn_create.
 *
 * attn_prefill / attn_decode on a shard context compute that shard's heads only:
 *  - cache_k, cache_v are the shard's own caches [B,S_max,n,128] (its kv heads);
 *  - attn_debug_buffers' q_r and h are [B*T,512 n];
 *  - delta receives the shard's PARTIAL Delta_attn [B,T,4096] fp32 = H_shard W_O_shard^T:
 *    the block's Delta_attn is the sum of the partials of all shards, which the row-parallel
 *    output projection's all-reduce (a sum over ranks, done by the caller, e.g. with
 *    torch.distributed.all_reduce) produces.
 * The residual forms (attn_set_norm, attn_*_residual) need the whole sum and return
 * GQA_ERR_INVALID_ARG on a shard context: apply attention_norm before the shards and add x
 * after the all-reduce.  n_kv_local = 8 gives the same context as attn_create.
 * Errors: those of attn_create, and GQA_ERR_SHAPE for n_kv_local outside 1..8.
 */
gqa_status attn_create_shard(const void *wq_shard, const void *wk_shard, const void *wv_shard,
                             const void *wo_shard, int n_kv_local, gqa_stream_t stream, gqa_ctx **out);

/*
 * attn_prefill — Delta_attn for T new positions of B sequences (steps 1-14).
 *
 * x       [B,T,4096] bf16: the block input, already normalised by the caller
 *         (the page's x_attn = attention_norm(x)).
 * R       [T,64,2] fp32: (cos, sin) of the rotation for positions start_pos+t,
 *         t = 0..T-1, pair j (the page's R [T positions, 64 pairs]).
 * causal  non-zero: M[t,s] = -inf for keys s > start_pos+t, else 0 (the quoted
 *         triu(diagonal=1) mask hstacked after start_pos zero columns); zero: M = 0.
 * cache_k, cache_v  [B,S_max,8,128] bf16 key / value cache.  Positions
 *         0..start_pos-1 must already hold rotated keys (cache_k) and values (cache_v)
 *         of the earlier positions; this call writes K_r and V of its T positions at
 *         start_pos..start_pos+T-1, then attends over keys 0..start_pos+T-1.  Other
 *         positions are neither read nor written.
 * delta   [B,T,4096] fp32 output, fully overwritten.
 * Requires B >= 1, T >= 1, start_pos >= 0, start_pos + T <= S_max, and
 * B*T <= 262144, S_max <= 1048576.
 * Intermediates (Q_r and H, bf16) live in the context's workspace, which grows on
 * demand: a call that needs a larger workspace synchronises `stream` and reallocates
 * (so the first call at a new maximum size is not capturable in a CUDA graph).
 */
gqa_status attn_prefill(gqa_ctx *ctx, const void *x, int B, int T, const float *R, int causal,
                        void *cache_k, void *cache_v, int S_max, int start_pos, float *delta,
                        gqa_stream_t stream);

/*
 * attn_decode — one new position per sequence (T = 1, no mask: every cached key is
 * visible, as in the quoted forward when seqlen == 1).
 *
 * x       [B,1,4096] bf16 block input of the new token of each sequence.
 * R_row   [1,64,2] fp32: rotation for position start_pos (shared by all sequences).
 * cache_k, cache_v  [B,S_max,8,128] bf16; positions 0..start_pos-1 hold the earlier
 *         rotated keys / values.  The new K_r, V are written at position start_pos,
 *         then the token attends over keys 0..start_pos.
 * delta   [B,1,4096] fp32 output.
 * Requires 1 <= B <= 1024, 0 <= start_pos < S_max <= 1048576.
 */
gqa_status attn_decode(gqa_ctx *ctx, const void *x, int B, int start_pos, const float *R_row,
                       void *cache_k, void *cache_v, int S_max, float *delta,
                       gqa_stream_t stream);

/*
 * The block's residual form.  The transformer block around this attention block computes
 * h = x + Delta_attn(attention_norm(x)) (page "Llama 3.1 8B · Merge and project", code
 * excerpt model.py 236-248 and "Contextual evidence from Output projection"), with
 * attention_norm an RMSNorm of weight w and eps = norm_eps = 1e-05 (sku_list.py arch_args on
 * the same page).  The pages do not print the RMSNorm body; it is read as
 *     attention_norm(x)[t, j] = x[t, j] / sqrt(mean_k x[t, k]^2 + eps) * w[j].
 * The library folds w into a second copy of W_Q, W_K, W_V (made by attn_set_norm) and scales
 * each token row of the projections by 1 / rms in their epilogue; the residual add happens in
 * the epilogue of the W_O projection.
 */

/*
 * attn_set_norm — give the context the attention_norm weight.
 *
 * norm_w  [4096] bf16 device tensor, read during this call only (the folded copy it makes,
 *         W_QKV * diag(norm_w) in bf16, 48 MiB, is owned by the context; a later call
 *         replaces it).
 * eps     the RMSNorm epsilon (> 0; 1e-5 for the Llama 3 / 3.1 8B configurations).
 * Enqueued on `stream`.  Errors: GQA_ERR_INVALID_ARG (null, eps <= 0 or not finite),
 * GQA_ERR_ALIGN, GQA_ERR_DEVICE, GQA_ERR_OOM, GQA_ERR_CUDA.
 */
gqa_status attn_set_norm(gqa_ctx *ctx, const void *norm_w, float eps, gqa_stream_t stream);

/*
 * attn_prefill_residual — h_out = x + Delta_attn(attention_norm(x)) for T new positions of
 * B sequences: attn_prefill with the normalisation in front and the residual add behind.
 *
 * x       [B,T,4096] bf16: the residual stream entering the block (not normalised).
 * h_out   [B,T,4096] fp32 output (x widened to fp32 plus Delta_attn), fully overwritten;
 *         it must not overlap x.
 * Every other argument, requirement and the cache semantics are those of attn_prefill.
 * Errors: those of attn_prefill, and GQA_ERR_INVALID_ARG when attn_set_norm has not been
 * called on the context.
 */
gqa_status attn_prefill_residual(gqa_ctx *ctx, const void *x, int B, int T, const float *R, int causal,
                                 void *cache_k, void *cache_v, int S_max, int start_pos, float *h_out,
                                 gqa_stream_t stream);

/*
 * attn_decode_residual — attn_decode in the residual form: x [B,1,4096] bf16 residual
 * stream of the new token of each sequence, h_out [B,1,4096] fp32 = x + Delta_attn
 * (must not overlap x).  Other arguments and errors as attn_decode, plus
 * GQA_ERR_INVALID_ARG when attn_set_norm has not been called on the context.
 */
gqa_status attn_decode_residual(gqa_ctx *ctx, const void *x, int B, int start_pos, const float *R_row,
                                void *cache_k, void *cache_v, int S_max, float *h_out,
                                gqa_stream_t stream);

/*
 * Drafted trees over a cache (speculative decoding).  A draft proposes T tokens per sequence
 * that form a tree: each token continues the prefix or another drafted token.  One call
 * verifies them all: the drafted tokens' keys and values lie behind the prefix, at positions
 * prefix_len[b] .. prefix_len[b] + T - 1, and token t sees the prefix and the drafted tokens
 * its mask row names (itself and its ancestors).
 */
#define GQA_MAX_TREE 256 /* drafted tokens per sequence */

/*
 * attn_tree_attention — the attention of T drafted tokens per sequence (head sharing, scores,
 * scaling, mask, softmax, value product, merge): for token t and query head h of kv head g
 *     h[b,t,h] = sum_s a_s v_s,  a = softmax over the visible s of q_r[b,t,h] . k_s / sqrt(128)
 * where s runs over positions 0 .. prefix_len[b] - 1 and prefix_len[b] + j for the bits j set
 * in row t of the mask.
 *
 * q_r     [B,T,512 n_kv] bf16: rotated queries (n_kv: the context's kv heads, 8 for the block).
 * tree_mask [B,T,ceil(T/32)] 32-bit words: bit j & 31 of word j / 32 of row (b, t) lets token t
 *         see drafted token j; bits at T and above are ignored.  A token without its own bit
 *         does not see itself; a row with no visible key at all gets zeros (so sequences with
 *         fewer drafted tokens are padded with empty rows).
 * cache_k, cache_v  [B,S_max,n_kv,128] bf16, read only.  Positions that no row sees may hold
 *         anything; the values of a drafted position that some row of the sequence sees have
 *         to be finite also for the rows that do not see it.
 * prefix_len [B] int32: 0 .. S_max - T.  Out of range: that sequence's rows of h are NaN and
 *         attn_sync_status reports GQA_ERR_SHAPE.
 * h       [B,T,512 n_kv] bf16 output, fully overwritten; must not overlap the inputs.
 * Requires 1 <= B <= 1024, 1 <= T <= GQA_MAX_TREE, T <= S_max <= 1048576.
 */
gqa_status attn_tree_attention(gqa_ctx *ctx, const void *q_r, int B, int T, const unsigned *tree_mask,
                               const void *cache_k, const void *cache_v, int S_max, const int *prefix_len,
                               void *h, gqa_stream_t stream);

/*
 * attn_prefill_tree — the block for a drafted tree: Delta_attn of T drafted tokens per
 * sequence.  Writes their K_r and V at positions prefix_len[b] + t, then attends as
 * attn_tree_attention does.
 *
 * x       [B,T,4096] bf16 block input of the drafted tokens.
 * R       [B,T,64,2] fp32: (cos, sin) for each token's own position (prefix_len[b] + its depth
 *         in the tree).
 * delta   [B,T,4096] fp32 output, fully overwritten (NaN for a sequence whose prefix_len is
 *         out of range; its cache is not written).
 * Other arguments, limits and the workspace as attn_tree_attention and attn_prefill.  On a
 * shard context delta is the shard's partial sum.
 * attn_prefill_tree_residual — the same in the residual form (see attn_prefill_residual).
 */
gqa_status attn_prefill_tree(gqa_ctx *ctx, const void *x, int B, int T, const float *R, const unsigned *tree_mask,
                             void *cache_k, void *cache_v, int S_max, const int *prefix_len, float *delta,
                             gqa_stream_t stream);
gqa_status attn_prefill_tree_residual(gqa_ctx *ctx, const void *x, int B, int T, const float *R,
                                      const unsigned *tree_mask, void *cache_k, void *cache_v, int S_max,
                                      const int *prefix_len, float *h_out, gqa_stream_t stream);

/*
 * attn_cache_commit — keep the accepted path of a verified tree: positions prefix_len[b] +
 * path[b,i] of both caches move to prefix_len[b] + i for i < n_accept[b], in place.
 *
 * path    [B,T] int32: drafted tokens of the accepted path, strictly increasing, each below T;
 *         entries from n_accept[b] on are not read.
 * n_accept [B] int32: 0 .. T.
 * new_len [B] int32 output: prefix_len[b] + n_accept[b]; may be the array prefix_len itself,
 *         but not overlap it otherwise, nor path or n_accept.
 * A sequence whose prefix_len, n_accept or path is out of range (or not increasing) is left as
 * it is, its new_len is its prefix_len, and attn_sync_status reports GQA_ERR_SHAPE.  Positions
 * behind the new length keep what they hold.  Limits as attn_tree_attention.
 */
gqa_status attn_cache_commit(gqa_ctx *ctx, void *cache_k, void *cache_v, int B, int S_max, int T,
                             const int *prefix_len, const int *path, const int *n_accept, int *new_len,
                             gqa_stream_t stream);

/*
 * Eviction by accumulated attention weight.  A decode step adds the softmax weight that each
 * key received, summed over the query heads of its kv head, to a running sum; when a cache has
 * grown past its budget, each kv head keeps its first and its most recent positions and the
 * heaviest of the others.  Keys keep the rotation of the position they were written for.
 * Only attn_decode_attention_weights and attn_decode_weights add weights: behind a prefill or
 * a verified tree the sums are what they were, and equal weights leave the lower positions.
 */

/*
 * attn_decode_attention_weights — decode attention (one query position per sequence over keys
 * 0 .. kv_len[b] - 1) that accumulates the key weights:
 *     weights[b,g,s] += sum over the 4 query heads of kv head g of their softmax weight on s.
 *
 * q_r     [B,512 n_kv] bf16; cache_k, cache_v [B,S_max,n_kv,128] bf16, read only.
 * kv_len  [B] int32: 0 .. S_max (0: h is zero).  Out of range: the sequence's h is NaN, its
 *         weights stay as they are, and attn_sync_status reports GQA_ERR_SHAPE.
 * weights [B,n_kv,S_max] fp32, updated at s < kv_len[b]; the other entries are not touched.
 * h       [B,512 n_kv] bf16 output; h and weights must not overlap the inputs or each other.
 * Requires 1 <= B <= 1024, 1 <= S_max <= 1048576.
 */
gqa_status attn_decode_attention_weights(gqa_ctx *ctx, const void *q_r, const void *cache_k, const void *cache_v,
                                         int B, int S_max, const int *kv_len, float *weights, void *h,
                                         gqa_stream_t stream);

/*
 * attn_decode_weights — the block for one new token per sequence, at cache position kv_len[b]
 * (0 .. S_max - 1): writes its K_r and V there, attends over keys 0 .. kv_len[b] and
 * accumulates their weights.  kv_len itself is not changed.
 *
 * x [B,1,4096] bf16; R [B,64,2] fp32: rotation of each sequence's new token (its position in
 * the text, which an eviction makes larger than kv_len[b]); delta [B,1,4096] fp32.
 * attn_decode_weights_residual — the same in the residual form (see attn_decode_residual).
 */
gqa_status attn_decode_weights(gqa_ctx *ctx, const void *x, int B, const float *R, void *cache_k, void *cache_v,
                               int S_max, const int *kv_len, float *weights, float *delta, gqa_stream_t stream);
gqa_status attn_decode_weights_residual(gqa_ctx *ctx, const void *x, int B, const float *R, void *cache_k,
                                        void *cache_v, int S_max, const int *kv_len, float *weights, float *h_out,
                                        gqa_stream_t stream);

/*
 * attn_cache_evict — cut every sequence to at most `budget` positions per kv head.  A sequence
 * with kv_len[b] <= budget keeps all its positions.  Otherwise each kv head keeps positions
 * 0 .. n_first - 1, the last n_recent, and of those between the budget - n_first - n_recent with
 * the largest weight (of equal weights the lower positions; a NaN counts less than any number).
 * What is kept moves to the front in ascending order, and its weights with it.
 *
 * cache_k, cache_v [B,S_max,n_kv,128] bf16, weights [B,n_kv,S_max] fp32, kv_len [B] int32.
 * out_k, out_v [B,S_out,n_kv,128], out_weights [B,n_kv,S_out]: the cut caches.  In place:
 *         the three inputs themselves with S_out = S_max; then positions from the new length
 *         on keep what they hold, and weights from the new length to the old one become 0.
 *         Otherwise no output may overlap an input, positions of out_k and out_v from the new
 *         length on are not written, and out_weights is 0 there.
 * kept    [B,n_kv,budget] int32 output: the position that each kept one had; -1 past the new
 *         length.
 * new_len [B] int32 output: min(kv_len[b], budget); may be the array kv_len itself, but not
 *         overlap it otherwise.  No output may overlap another.
 * Requires 1 <= budget <= S_out, n_first, n_recent >= 0, n_first + n_recent <= budget, and the
 * limits of attn_decode_attention_weights.  A kv_len outside 0 .. S_max: the sequence's caches
 * and weights stay as they are, its kept is -1, its new_len 0, and attn_sync_status reports
 * GQA_ERR_SHAPE.
 */
gqa_status attn_cache_evict(gqa_ctx *ctx, const void *cache_k, const void *cache_v, const float *weights, int B,
                            int S_max, const int *kv_len, int budget, int n_first, int n_recent, void *out_k,
                            void *out_v, float *out_weights, int S_out, int *kept, int *new_len,
                            gqa_stream_t stream);

/*
 * Paged caches.  A server that shares one pool of cache memory among its sequences hands it out in
 * pages of page_size positions; a page table names the pages of each sequence in order.  Position s
 * of sequence b is slot s % page_size of page page_table[b, s / page_size].  Three steps use it:
 * attn_rope_apply rotates queries, attn_paged_append rotates keys and writes them and the values to
 * their pages, attn_paged_decode_attention attends with one new token per sequence;
 * attn_decode_paged is the whole block over such a cache.
 */

/* Which elements of a head are rotated together by pair j of rot_dim / 2; elements from rot_dim on
 * are not rotated. */
enum {
    GQA_ROPE_PAIRS = 0, /* (2j, 2j + 1), as the block's projections do */
    GQA_ROPE_HALVES = 1 /* (j, j + rot_dim / 2) */
};

/* How the frequencies w_j = theta^(-2j / rot_dim) are scaled for contexts longer than the model was
 * trained with. */
enum {
    GQA_ROPE_PLAIN = 0,  /* not at all */
    GQA_ROPE_LINEAR = 1, /* w / factor */
    GQA_ROPE_BANDS = 2,  /* by wavelength 2 pi / w: shorter than context / high keeps w, longer than context / low
                            takes w / factor, and in between (1 - m) w / factor + m w with
                            m = (context / wavelength - low) / (high - low) */
    GQA_ROPE_RAMP = 3    /* m w / factor + (1 - m) w, m = clamp((j - a) / (b - a), 0, 1); a and b are the pairs that
                            turn `high` and `low` times over the context, pair(n) =
                            rot_dim ln(context / (2 pi n)) / (2 ln theta), a = max(floor pair(high), 0),
                            b = min(ceil pair(low), rot_dim - 1) (b - a: at least 0.001); the rotated part
                            is multiplied by gain = 0.1 ln(factor) + 1 */
};

typedef struct {
    int kind;                          /* GQA_ROPE_PLAIN .. GQA_ROPE_RAMP */
    double factor, low, high, context; /* those that the kind does not use are not read */
} gqa_rope_scaling;

/* A rotation, filled in by attn_rope_init and kept by the caller (host memory, no pointers in it:
 * may be copied).  turns[j]: revolutions per position of pair j, as a fraction of 2^64. */
typedef struct {
    unsigned long long turns[64];
    float gain;
    int layout, rot_dim, check;
} gqa_rope;

/*
 * attn_rope_init — set up a rotation (host only; needs no GPU).  layout as above; rot_dim a
 * multiple of 16 in 16 .. 128; theta > 1; scaling may be NULL (GQA_ROPE_PLAIN).
 * Pair j at position p turns by p turns[j] / 2^64 revolutions, an exact integer product of which the
 * whole revolutions fall away: far positions lose nothing to the size of the angle.
 * Errors: GQA_ERR_INVALID_ARG (null; layout or kind unknown; a parameter not finite or out of
 * range: theta > 1, factor >= 1, context > 0, 0 < low < high), GQA_ERR_SHAPE (rot_dim).
 */
gqa_status attn_rope_init(gqa_rope *rope, int layout, int rot_dim, double theta, const gqa_rope_scaling *scaling);

/*
 * attn_rope_apply — rotate n_heads heads of n_tok tokens: (a, b) of pair j becomes
 * gain (a cos - b sin, a sin + b cos) of the angle of positions[t], in fp32, rounded once.
 *
 * x       bf16: head h of token t at x + t stride + 128 h (elements); rows of a fused projection
 *         may be given as they are.
 * positions [n_tok] int32, any value (a negative one turns backwards).
 * out     bf16, the same form with its own stride; x itself with the same stride rotates in
 *         place, otherwise its memory from the first to the last row must not overlap x's.
 * Requires 1 <= n_tok <= 262144, 1 <= n_heads <= 1024, both strides multiples of 8 and at least
 * 128 n_heads (and below 2^31).
 */
gqa_status attn_rope_apply(gqa_ctx *ctx, const gqa_rope *rope, const void *x, int n_tok, int n_heads,
                           long long stride, const int *positions, void *out, long long out_stride,
                           gqa_stream_t stream);

/*
 * attn_rope_table — the table R [n_tok,64,2] fp32 of (cos, sin) that the block forms take, for
 * positions[t] [n_tok] int32; pairs from rot_dim / 2 on are (1, 0).  1 <= n_tok <= 262144.
 * A rotation in halves has no such table (GQA_ERR_INVALID_ARG).
 */
gqa_status attn_rope_table(gqa_ctx *ctx, const gqa_rope *rope, const int *positions, int n_tok, float *R,
                           gqa_stream_t stream);

enum {
    GQA_CACHE_BF16 = 0, /* bfloat16 */
    GQA_CACHE_E4M3 = 1  /* 8-bit floating point (4 exponent bits, 3 mantissa bits) times a scale per kv head */
};

typedef struct gqa_paged gqa_paged; /* opaque */

/*
 * attn_paged_create — describe the two pools of a paged cache for the context's kv heads (host only,
 * enqueues nothing).  Element d of head g in slot i of page n is at
 *     n stride_page + i stride_pos + g stride_head + d    (elements),
 * so [page, slot, head, 128], [page, head, slot, 128] and pools that keep a page's keys and values
 * side by side are all described.
 *
 * k_pages, v_pages  the pools, owned by the caller; they must outlive the description.
 * dtype   GQA_CACHE_BF16 or GQA_CACHE_E4M3.
 * strides multiples of 16 bytes, and each at least what all smaller ones reach together with the row of 128
 *         elements, so that no two rows overlap; the stride of an extent of 1 is not read.  No key's row may
 *         overlap a value's (the pools may lie in one another's gaps).
 * k_scale, v_scale  GQA_CACHE_E4M3: [n_kv] fp32 on the device, positive and normal: a key or value is the
 *         stored number times its head's scale (NULL: 1).  Read by every call that uses the pools.
 *         A key scale that is negative, infinite or NaN makes its heads' results NaN.
 *         NULL for bf16.
 * Requires n_pages >= 1, page_size a multiple of 8 in 8 .. 1048576, strides below 2^39 bytes
 * and pools that span at most 2^46 elements.
 * Errors: GQA_ERR_INVALID_ARG (null, dtype unknown, scales with bf16, rows that overlap, the same
 * pool twice), GQA_ERR_SHAPE, GQA_ERR_ALIGN, GQA_ERR_OOM, GQA_ERR_CUDA.
 * A description may be used with any context of as many kv heads on the same device.
 */
gqa_status attn_paged_create(gqa_ctx *ctx, void *k_pages, void *v_pages, int n_pages, int page_size, int dtype,
                             long long stride_page, long long stride_pos, long long stride_head,
                             const float *k_scale, const float *v_scale, gqa_paged **out);

/* attn_paged_destroy — free a description (not the pools).  Work that is enqueued does not need it.
 * NULL is ignored. */
void attn_paged_destroy(gqa_paged *paged);

/*
 * attn_paged_append — write n_new[b] new positions of each sequence behind its kv_len[b]:
 *     K[kv_len[b] + t] = rotation of k[b,t],  V[kv_len[b] + t] = v[b,t],  t < n_new[b].
 * The rotation is in fp32 and rounded once to the pools' type (e4m3: times the reciprocal of the
 * head's scale, saturating at 448; a NaN stays one).
 *
 * k, v    bf16: head g of token t of sequence b at b stride_b + t stride_t + 128 g (elements): rows of
 *         a fused projection, or a dense cache [B,S_max,n_kv,128] that attn_prefill has filled.
 *         Strides multiples of 8, at least 128 n_kv and below 2^31; stride_b is not read for B = 1, nor
 *         stride_t for T = 1.  From their first to their last row they must not overlap the memory from a
 *         pool's first to its last row.
 * rope    the rotation; NULL: keys are written as they are (already rotated).
 * rope_pos [B] int32: position of each sequence's first new token in its text; NULL: kv_len[b].
 * page_table [B,max_pages] int32; entries of pages that hold no new position are not read.
 * kv_len  [B] int32; not changed by the call.
 * n_new   [B] int32: 0 .. T, or NULL: T for every sequence; k and v from n_new[b] on are not read.
 * A sequence with n_new[b] outside 0 .. T, or kv_len[b] outside 0 .. max_pages page_size -
 * n_new[b], is left out, and so are positions whose page is outside 0 .. n_pages - 1;
 * attn_sync_status then reports GQA_ERR_SHAPE.  No two new positions may share a slot.
 * Requires 1 <= B <= 1024, T >= 1, B T <= 262144, 1 <= max_pages, max_pages page_size <= 1048576.
 */
gqa_status attn_paged_append(gqa_ctx *ctx, const gqa_paged *paged, const void *k, const void *v, int B, int T,
                             long long stride_b, long long stride_t, const gqa_rope *rope, const int *rope_pos,
                             const int *page_table, int max_pages, const int *kv_len, const int *n_new,
                             gqa_stream_t stream);

/*
 * attn_paged_decode_attention — attention of one query position per sequence over keys 0 ..
 * kv_len[b] - 1 of a paged cache.
 *
 * q_r     [B,512 n_kv] bf16 rotated queries.
 * page_table [B,max_pages] int32; entries from ceil(kv_len[b] / page_size) on are not read, and
 *         neither are slots from kv_len[b] on.  Sequences may share pages.
 * kv_len  [B] int32: 0 .. max_pages page_size (0: h is zero).  Out of range, or with a page outside
 *         0 .. n_pages - 1 among those it reads: the sequence's h is NaN and attn_sync_status reports
 *         GQA_ERR_SHAPE.
 * h       [B,512 n_kv] bf16 output; must not overlap the inputs, the pools' rows and scales among them.
 * Limits as attn_paged_append.  The scratch (at most 2 MB) is the context's: the first call on it may allocate, and then
 * cannot be captured.
 */
gqa_status attn_paged_decode_attention(gqa_ctx *ctx, const gqa_paged *paged, const void *q_r, int B,
                                       const int *page_table, int max_pages, const int *kv_len, void *h,
                                       gqa_stream_t stream);

/*
 * attn_decode_paged — the block for one new token per sequence over a paged cache, at position
 * kv_len[b] (0 .. max_pages page_size - 1): writes its K_r and V to their page, attends over keys
 * 0 .. kv_len[b].  kv_len itself is not changed.
 *
 * x [B,1,4096] bf16; R [B,64,2] fp32: rotation of each sequence's new token (attn_rope_table);
 * delta [B,1,4096] fp32 (NaN for a sequence whose kv_len or a page is out of range; its cache is
 * not written where the new position's page is).  With an e4m3 cache the new key and value are rounded to
 * bf16 and then to e4m3.
 * attn_decode_paged_residual — the same in the residual form (see attn_decode_residual).
 */
gqa_status attn_decode_paged(gqa_ctx *ctx, const gqa_paged *paged, const void *x, int B, const float *R,
                             const int *page_table, int max_pages, const int *kv_len, float *delta,
                             gqa_stream_t stream);
gqa_status attn_decode_paged_residual(gqa_ctx *ctx, const gqa_paged *paged, const void *x, int B, const float *R,
                                      const int *page_table, int max_pages, const int *kv_len, float *h_out,
                                      gqa_stream_t stream);

/*
 * attn_sync_status — synchronise `stream`, then read and clear the context's device
 * status word.  Returns GQA_OK, GQA_ERR_TIMEOUT (a bounded device wait ran out in some
 * earlier call), GQA_ERR_SHAPE (a per-sequence length or path of some earlier call was out
 * of range; GQA_ERR_TIMEOUT comes first where both happened) or GQA_ERR_CUDA (the
 * synchronisation itself failed).
 */
gqa_status attn_sync_status(gqa_ctx *ctx, gqa_stream_t stream);

/*
 * attn_debug_buffers — device pointers to the context's intermediates after the last
 * call on it: q_r [B*T,4096] bf16 (rotated queries) and h [B*T,4096] bf16 (merged head
 * outputs, the page's H after step 13).  Valid until the next call on the context.
 * Either out-pointer may be NULL.  Returns GQA_ERR_INVALID_ARG for a null context.
 */
gqa_status attn_debug_buffers(gqa_ctx *ctx, const void **q_r, const void **h);

/*
 * Per-kernel device timing (tracing).  Kernel kinds:
 */
enum {
    GQA_KERNEL_QKV_GEMM = 0,       /* fused Q/K/V projection + RoPE + cache write (many tokens) */
    GQA_KERNEL_QKV_SPLITK = 1,     /* the same for few tokens: cluster split-K with its reduction */
    GQA_KERNEL_FLASH_PREFILL = 2,  /* causal GQA attention, prefill */
    GQA_KERNEL_DECODE_ATTN = 3,    /* split-KV attention with the fused merge, decode */
    GQA_KERNEL_OUT_GEMM = 4,       /* Delta = H W_O^T (many tokens) */
    GQA_KERNEL_OUT_SPLITK = 5,     /* the same for few tokens */
    GQA_KERNEL_RMS_NORM = 6,       /* 1 / rms of each token row (residual form only) */
    GQA_KERNEL_CACHE_ATTN = 7,     /* tree attention / decode attention with key weights */
    GQA_KERNEL_CACHE_MERGE = 8,    /* its merge of sequences that several workers share */
    GQA_KERNEL_CACHE_WEIGHTS = 9,  /* with key weights: the merge and their accumulation */
    GQA_KERNEL_CACHE_COMMIT = 10,  /* accepted path moved behind the prefix */
    GQA_KERNEL_EVICT_SELECT = 11,  /* positions that an eviction keeps */
    GQA_KERNEL_EVICT_MOVE = 12,    /* their keys and values moved */
    GQA_KERNEL_PAGED_ATTN = 13,    /* decode attention over a paged cache, with its merge */
    GQA_KERNEL_PAGED_APPEND = 14,  /* new keys (rotated) and values written to their pages */
    GQA_KERNEL_ROPE = 15,          /* rotation of queries, or the table of a rotation */
    GQA_KERNEL_KINDS = 16
};

/*
 * attn_profile_begin — from now on, every kernel this context launches is bracketed by
 * two CUDA events recorded on the launch stream (up to 65536 launches).  Recording adds
 * two event records per launch and nothing else.
 * attn_profile_end_kinds — stop recording, synchronise `stream`, and write, for the first
 * n_kinds kernel kinds, the summed device time in milliseconds (ms_per_kind[n_kinds]) and the
 * number of launches (launches_per_kind[n_kinds]) since attn_profile_begin; 0 for kinds that
 * this library does not have.  Either output may be NULL.  Errors: GQA_ERR_INVALID_ARG (null
 * context, n_kinds < 0), GQA_ERR_CUDA.
 * attn_profile_end — the same for all GQA_KERNEL_KINDS kinds of the header that a program is
 * built with.  The library's function of that name writes the first seven kinds, which is what
 * the arrays of programs built before there were more hold.
 */
gqa_status attn_profile_begin(gqa_ctx *ctx);
gqa_status attn_profile_end_kinds(gqa_ctx *ctx, double *ms_per_kind, int *launches_per_kind, int n_kinds,
                                  gqa_stream_t stream);
gqa_status attn_profile_end(gqa_ctx *ctx, double *ms_per_kind, int *launches_per_kind,
                            gqa_stream_t stream);
#define attn_profile_end(ctx, ms_per_kind, launches_per_kind, stream) \
    attn_profile_end_kinds(ctx, ms_per_kind, launches_per_kind, GQA_KERNEL_KINDS, stream)

/*
 * attn_decode_attention_noalloc — the decode attention of attn_decode (key/value head
 * sharing, scores, scaling, softmax over keys 0..kv_len-1, value product, head merge) for
 * callers that cannot let this library allocate device memory.  The pages have no
 * counterpart for this entry point: it exists for a serving engine that keeps all of HBM
 * in its own pool (for example for a paged KV cache) and gives a library only its inputs
 * and outputs, and for decode loops that cannot afford the device-wide synchronisation a
 * cudaMalloc implies.  It allocates nothing and needs no context.
 *
 * q_r     [B,4096] bf16: rotated queries of the new token of each sequence (what
 *         attn_debug_buffers returns as q_r after attn_decode).
 * cache_k, cache_v  [B,S_max,8,128] bf16: rotated keys / values; positions 0..kv_len-1
 *         are read (the new token's entry must already be written), nothing is written.
 * h       [B,4096] bf16 output: merged head outputs (the page's H after the merge).
 * Limits: 1 <= B <= 256, 1 <= kv_len <= S_max <= 1048576; larger B returns GQA_ERR_SHAPE.
 *
 * Scratch: the per-split partial results live in one file-scope device array of about
 * 4.3 MB (2048 units of (sequence, kv head, key split)), which every GPU that loads this
 * library holds until the process exits.  The first call on a device looks up that
 * array's device address (cudaGetSymbolAddress), the device's SM count and architecture,
 * and configures the kernels; make that first call before any stream capture.  Every call
 * shares the array and it keeps the last call's contents; calls whose work overlaps on the
 * GPU (other streams or host threads) race and must be serialised by the caller.
 * Time-outs: if a bounded device-side wait of this call runs out, every element of h is
 * written as NaN (never a mix of stale partial results) and the time-out is recorded in a
 * status word inside the array, which attn_decode_attention_noalloc_status reports.
 * Errors: GQA_ERR_INVALID_ARG, GQA_ERR_SHAPE, GQA_ERR_ALIGN, GQA_ERR_DEVICE (not sm_103),
 * GQA_ERR_CUDA (the cause via attn_last_cuda_error).
 */
gqa_status attn_decode_attention_noalloc(const void *q_r, const void *cache_k,
                                         const void *cache_v, int B, int kv_len, int S_max,
                                         void *h, gqa_stream_t stream);

/*
 * attn_decode_attention_noalloc_status — synchronise `stream`, then read and clear the
 * status word of attn_decode_attention_noalloc on the current device (allocates nothing).
 * Returns GQA_ERR_TIMEOUT if a device-side wait of any call since the last read ran out
 * (those calls wrote NaN into their h), GQA_OK otherwise, or GQA_ERR_DEVICE / GQA_ERR_CUDA.
 * The word is shared by every caller of the entry point on that device.
 */
gqa_status attn_decode_attention_noalloc_status(gqa_stream_t stream);

/*
 * attn_decode_attention_noalloc_debug_inject_timeout — test hook for that failure path (no
 * counterpart on the pages): the next call of attn_decode_attention_noalloc (in any thread)
 * makes its first work unit issue no loads, so that unit's bounded waits run out after about
 * 2 s; nothing faults or hangs.  Always returns GQA_OK.
 */
gqa_status attn_decode_attention_noalloc_debug_inject_timeout(void);

/*
 * attn_debug_inject_timeout — test hook for the failure path (no counterpart on the pages).
 * Arms a one-shot flag: on the next launch of kernel kind `kind` (GQA_KERNEL_QKV_GEMM,
 * _QKV_SPLITK, _FLASH_PREFILL, _DECODE_ATTN, _OUT_GEMM, _OUT_SPLITK, _CACHE_ATTN or _PAGED_ATTN) made through this
 * context, the first work unit's (_CACHE_ATTN, _PAGED_ATTN: the last worker's) TMA producer issues no loads.  Its consumers' bounded
 * waits then run out (about 2 s), the unit records GQA_ERR_TIMEOUT in the status word,
 * releases its tensor memory and returns; kernels queued after it on the stream may time
 * out too.  Nothing faults or hangs.  The outputs of that call are undefined; the next
 * attn_sync_status returns GQA_ERR_TIMEOUT and resets the device-side state, after which
 * the context is usable again.  Errors: GQA_ERR_INVALID_ARG (null context, other kind).
 */
gqa_status attn_debug_inject_timeout(gqa_ctx *ctx, int kind);

/*
 * attn_debug_pair_schedule — the work schedule of the many-token projection GEMM, computed
 * on the host exactly as the library sizes a launch and as each CTA pair walks it (no
 * counterpart on the pages; for tests, no GPU needed).  Output tiles of 256 x 256:
 * m_tiles x n_tiles of them (n_tiles 24 for the Q/K/V projection, 16 for W_O), over n_pairs
 * co-resident CTA pairs.  Writes *full_rounds (rounds of whole tiles), *tail_w (width of the
 * pieces the last, partial round is cut into; 0: none) and *grid_ctas (CTAs launched), and
 * the items in launch order of pairs, each pair's items in the order it runs them, as
 * quadruples (pair, m tile, first column, width) into items[4 * max_items]; *n_items gets
 * their count.  Errors: GQA_ERR_INVALID_ARG (null pointer, m_tiles, n_tiles or n_pairs < 1,
 * max_items < 0), GQA_ERR_SHAPE (more than max_items items; *n_items holds the count).
 */
gqa_status attn_debug_pair_schedule(int m_tiles, int n_tiles, int n_pairs, int *full_rounds,
                                    int *tail_w, int *grid_ctas, int *items, int max_items,
                                    int *n_items);

/*
 * attn_debug_cache_schedule — how tree attention and attn_decode_attention_weights share the
 * 128-key tiles of B sequences among `workers` workers (CTAs or their softmax slots), computed
 * on the host by the code that the kernel runs (for tests, no GPU needed).  lens [B] (host), n_new
 * keys behind each length, units (kv heads x groups of query rows) per sequence, unit_cost (0 .. 64)
 * the tiles that beginning and ending a unit counts for (8, 3 and 2 in the kernels), workers 1 .. 32768.  Writes the
 * pieces in order as octuples (worker, sequence, unit, first tile, tiles, slot of its partial
 * result or -1 for a whole unit, last worker of the unit, number of the first tile among all
 * tiles) into pieces[8 * max_pieces]; *n_pieces gets their count.  Errors:
 * GQA_ERR_INVALID_ARG, GQA_ERR_SHAPE (more than max_pieces pieces; *n_pieces holds the count).
 */
gqa_status attn_debug_cache_schedule(const int *lens, int B, int n_new, int S_max, int units, int unit_cost,
                                     int workers, int *pieces, int max_pieces, int *n_pieces);

/*
 * attn_debug_exp2 — the two exponentials the prefill softmax uses, on n fp32 device inputs a
 * (no counterpart on the pages; for tests): out_fma[i] = 2^a[i] by the FMA-pipe cubic
 * (range reduction, a minimax cubic fitted for relative error, exponent insertion; inputs
 * below -125 give 2^-125) and out_mufu[i] = ex2.approx.ftz(a[i]), both fp32 device arrays of
 * n elements.  Enqueued on `stream`.  Errors: GQA_ERR_INVALID_ARG (null, n < 1), GQA_ERR_CUDA.
 */
gqa_status attn_debug_exp2(const float *a, float *out_fma, float *out_mufu, int n, gqa_stream_t stream);

/* attn_destroy — free everything the context owns (after synchronising the device).
 * NULL is ignored. */
void attn_destroy(gqa_ctx *ctx);

/* attn_strerror — static description of a status code (never NULL). */
const char *attn_strerror(gqa_status status);

/* attn_last_cuda_error — the cudaError_t value of the last failing CUDA call made by
 * this library on the calling thread (0 if none). */
int attn_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* GQA_ATTN_H */
