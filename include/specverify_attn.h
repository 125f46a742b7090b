/*
 * specverify_attn.h - the part of libspecverify.so's C ABI that works on the
 * model's side of a verification step: rotary positions, a paged cache of
 * keys and values, and the attention of each request's new tokens over it.
 *
 * One verification step of a request with K drafts runs the target model over
 * K + 1 new tokens (the last emitted token and the drafts).  In every layer
 * their queries and keys are turned by their positions, the keys and values
 * join the request's cache (sv_kv_append), and the new tokens attend to all
 * that the cache holds (sv_paged_attention).  The resulting logits go to
 * sv_spec_verify (specverify.h); after it the request's cache is kept up to
 * the accepted drafts by lowering its length, and the next step's append
 * overwrites the rest.  A chunk of a prompt is the same call with more new
 * tokens; a decoding step is the same call with one.
 *
 * The conventions of specverify.h hold: device memory is the caller's, work
 * is enqueued on `stream` without a host synchronisation, host checks come
 * first and a negative sv_status means nothing was launched, outputs are a
 * deterministic function of the inputs.  The calls keep no state: a workspace
 * holds nothing from one call to the next and needs no clearing, and any two
 * calls may run concurrently if they share no output and no workspace.  Calls
 * may be captured in HIP graphs.  The device that `stream` belongs to has to
 * be current.
 *
 * Packed sequences.  T rows (new tokens) are packed one request after
 * another: request b's rows are query_start[b] .. query_start[b+1] - 1
 * (int32 [B + 1], ascending).  Rows before query_start[0] and from
 * query_start[B] on belong to no request: no call writes any output of them.
 * A request may have no rows.
 *
 * Places.  kv_len[b] (int32 [B]) is the number of tokens of request b in the
 * cache, its new ones included: row i of its n rows is at place
 * kv_len[b] - n + i (a negative kv_len counts as 0).  Rows at negative places
 * are not stored and see nothing.
 */
#ifndef SPECVERIFY_ATTN_H
#define SPECVERIFY_ATTN_H

#include "specverify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of a cache: SV_BF16, or 8-bit floating point (1 sign, 4
 * exponent, 3 mantissa bits, largest value 448, no infinities) with one
 * power-of-two scale per token and head. */
#define SV_E4M3 2

/* Largest head size, heads, page size, tokens of a page table's row, and rows
 * of a call. */
#define SV_ATTN_MAX_HEAD_DIM 256
#define SV_ATTN_MAX_HEADS 1024
#define SV_ATTN_MAX_PAGE 65536
#define SV_ATTN_MAX_TOKENS 1073741824
#define SV_ATTN_MAX_ROWS (1 << 23)

/* A paged cache of keys and values, with the page table of the requests of a
 * call.  The token at place p of request b has its key at
 *   k + page * k_page_stride + (p % page_size) * k_token_stride
 *     + head * k_head_stride,   page = page_table[b * page_table_stride
 *                                                 + p / page_size]
 * (strides in elements, channels contiguous), its value likewise.  Pages and
 * heads may be laid out in any order; a token's rows may not overlap others.
 * A page outside 0..num_pages-1 and a place from max_pages * page_size on hold
 * nothing: what is written there is dropped, what is read there is absent
 * (sv_kv_gather writes zeros, sv_paged_attention does not see the token).
 * Requests may share pages that a call only reads; a token's rows may be
 * written by one row of a call only. */
typedef struct {
  int dtype;       /* SV_BF16 or SV_E4M3                                    */
  int heads;       /* key / value heads                                     */
  int head_dim;    /* a multiple of 16, 16..SV_ATTN_MAX_HEAD_DIM            */
  int page_size;   /* tokens of a page, a power of two                      */
  int num_pages;   /* pages of k and of v                                   */
  int max_pages;   /* entries of a page table's row                         */
  const int32_t* page_table;
  int64_t page_table_stride; /* entries between requests' rows, >= max_pages
                                (0: all requests share one row)             */
  void* k;         /* 16-byte aligned; strides multiples of 16 bytes        */
  void* v;
  int64_t k_page_stride, k_token_stride, k_head_stride;
  int64_t v_page_stride, v_token_stride, v_head_stride;
  uint8_t* k_scale; /* SV_E4M3: uint8 [num_pages, heads, page_size], the    */
  uint8_t* v_scale; /* biased exponent e + 127 of each row's scale 2^e (255: */
                    /* the row is NaN); SV_BF16: not read, may be NULL      */
} sv_paged_cache;

/* Layouts of the turned channels: pair i of `rotary_dim / 2` is channels
 * (i, i + rotary_dim / 2) or (2 i, 2 i + 1). */
typedef enum { SV_ROPE_HALF = 0, SV_ROPE_INTERLEAVED = 1 } sv_rope_layout;

/* How the frequencies are changed for contexts `factor` times the length
 * `original_len` that the model was trained at. */
typedef enum {
  SV_ROPE_PLAIN = 0,  /* f_i = base^(-2 i / rotary_dim), radians a position  */
  SV_ROPE_LINEAR = 1, /* f_i / factor                                        */
  SV_ROPE_BASE = 2,   /* base replaced by base * factor^(d / (d - 2))        */
  SV_ROPE_RAMP = 3,   /* from f_i to f_i / factor along a ramp over the pair
                         index, between the pairs that turn `high` and `low`
                         times over original_len (Peng et al. 2023, in the
                         form by channel index), and mscale 0.1 ln(factor)+1 */
  SV_ROPE_BANDS = 4   /* the same along a ramp over the number of turns
                         itself, mscale 1                                    */
} sv_rope_scaling;

/* The frequencies of rotary positions: host arithmetic in binary64.
 * freq: host, [rotary_dim / 2].  mscale: host, 1 value, the factor of cos and
 * sin.  factor >= 1; original_len > 0 and 0 < low < high turns are read by
 * SV_ROPE_RAMP and SV_ROPE_BANDS.  Returns SV_OK or SV_ERR_INVALID_ARG. */
int sv_rope_frequencies(int rotary_dim, double base, int scaling, double factor, double original_len, double low,
                        double high, double* freq, float* mscale);

/* Rotary positions: out = x with each pair (a, c) of the first rotary_dim
 * channels of every head replaced by
 *   mscale * (a cos t - c sin t, a sin t + c cos t),   t = positions[row] * freq[i],
 * the other channels copied; with backward != 0 by the transpose of that map
 * (t replaced by -t): the gradient with respect to x from the gradient with
 * respect to out.
 *   x, out     elements of type dtype (SV_F32 or SV_BF16), [T, heads,
 *              head_dim] with the given strides (elements) between rows and
 *              heads, channels contiguous; any alignment of whole elements.
 *              out may be x itself with the same strides; else they may not
 *              overlap.
 *   positions  int64 [T], |position| < 2^40.
 *   freq       binary64 [rotary_dim / 2] (device).
 * Angles are formed and reduced in binary64, cos and sin and the products in
 * binary32, the result rounded once.  head_dim 1..SV_ATTN_MAX_HEAD_DIM,
 * rotary_dim even, 0..head_dim. */
int sv_rope(void* stream, int T, int heads, int head_dim, int rotary_dim, int layout, int backward, int dtype,
            const void* x, int64_t x_token_stride, int64_t x_head_stride, const int64_t* positions,
            const double* freq, float mscale, void* out, int64_t out_token_stride, int64_t out_head_stride);

/* Appends the new tokens of B requests to a paged cache; see "Packed
 * sequences" and "Places" above.  The cache holds kv_len[b] tokens of request
 * b afterwards; what it held at the new tokens' places is overwritten.
 *   k, v       new keys and values, SV_F32 or SV_BF16 (dtype), [T,
 *              cache->heads, head_dim] with the given strides.
 *   q, q_out   NULL, or the new queries [T, q_heads, head_dim] of the same
 *              type and where they go once turned (q_out may be q itself with
 *              the same strides; q_heads 0 with NULL).
 *   freq       binary64 [rotary_dim / 2], or NULL (rotary_dim 0): keys and
 *              queries are not turned.
 *   positions  NULL: a row's position is its place; else int64 [T].
 * Keys are turned as by sv_rope in binary32 and rounded once, to the cache's
 * type.  SV_E4M3: with a the largest finite magnitude of the row, its scale is
 * the least power of two 2^e, -117 <= e <= 127, with a <= 448 * 2^e (e = -9
 * for a row of zeros), and each element is x / 2^e rounded to nearest even; an
 * element that is not finite is stored as NaN.  (From e = -117 on every value
 * the row can stand for is exact in bf16.) */
int sv_kv_append(void* stream, int B, int T, int q_heads, int dtype, int rotary_dim, int layout, const double* freq,
                 float mscale, const int64_t* positions, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                 void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride, const void* k,
                 int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
                 int64_t v_head_stride, const int32_t* query_start, const int32_t* kv_len,
                 const sv_paged_cache* cache);

/* Norms of query and key heads with their rotary positions in one pass: each
 * head's row x becomes rope(x * r * w), r = (mean of x^2 over head_dim +
 * eps)^-1/2, w the weights of queries or of keys, rope as by sv_rope (which
 * says what layouts, strides and positions may be).
 *   q, k, q_out, k_out   SV_F32 or SV_BF16 (dtype), [T, q_heads or k_heads,
 *              head_dim] with the given strides; an output may be its input
 *              with the same strides, else none may overlap another array.
 *              Heads 0: there are no queries, or no keys.
 *   q_weight, k_weight   [head_dim], SV_F32 or SV_BF16 (weight_dtype); NULL:
 *              all 1.
 *   eps        at least 2^-126, finite.
 *   positions  int64 [T]; not read with rotary_dim 0.
 * The sum of squares and all products are binary32, the result is rounded once:
 * a row whose sum of squares passes 3.4e38 has no meaningful result. */
int sv_qk_norm_rope(void* stream, int T, int q_heads, int k_heads, int head_dim, int rotary_dim, int layout, int dtype,
                    const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
                    int64_t k_token_stride, int64_t k_head_stride, int weight_dtype, const void* q_weight,
                    const void* k_weight, float eps, const int64_t* positions, const double* freq, float mscale,
                    void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride, void* k_out,
                    int64_t k_out_token_stride, int64_t k_out_head_stride);

/* Bytes of workspace that sv_qk_norm_rope_backward needs where a weight's
 * gradient is asked for; 0 for sizes that the call would reject. */
size_t sv_qk_norm_rope_backward_workspace_size(int T, int head_dim);

/* The gradients of sv_qk_norm_rope: from dq_out, dk_out (with respect to its
 * outputs; type and shape as q, k) those with respect to q, k and the weights.
 *   dq, dk     as q, k; each may be its dq_out or q (dk_out or k) with the same
 *              strides.
 *   dq_weight, dk_weight   float [head_dim] (also where the weights themselves
 *              are NULL), or NULL: not asked for.  Sums over rows and heads in
 *              binary32, in an order that depends on T alone; 0 with T == 0.
 *   workspace  scratch of this call alone, 16-byte aligned; NULL where neither
 *              weight's gradient is asked for. */
int sv_qk_norm_rope_backward(void* stream, int T, int q_heads, int k_heads, int head_dim, int rotary_dim, int layout,
                             int dtype, const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
                             int64_t k_token_stride, int64_t k_head_stride, const void* dq_out,
                             int64_t dq_out_token_stride, int64_t dq_out_head_stride, const void* dk_out,
                             int64_t dk_out_token_stride, int64_t dk_out_head_stride, int weight_dtype,
                             const void* q_weight, const void* k_weight, float eps, const int64_t* positions,
                             const double* freq, float mscale, void* dq, int64_t dq_token_stride,
                             int64_t dq_head_stride, void* dk, int64_t dk_token_stride, int64_t dk_head_stride,
                             float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes);

/* sv_kv_append with norms: keys and queries are normed before they are turned,
 * values are not.  Queries are formed in binary32 as by sv_qk_norm_rope and
 * rounded once.  Keys, which every later row reads, are formed in binary64, from
 * finite rows of any size, and rounded once to SV_E4M3, to SV_BF16 by way of
 * binary32.  Both may differ by these roundings from what sv_qk_norm_rope gives. */
int sv_kv_append_normed(void* stream, int B, int T, int q_heads, int dtype, int rotary_dim, int layout,
                        const double* freq, float mscale, const int64_t* positions, int weight_dtype,
                        const void* q_weight, const void* k_weight, float eps, const void* q, int64_t q_token_stride,
                        int64_t q_head_stride, void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                        const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                        int64_t v_token_stride, int64_t v_head_stride, const int32_t* query_start,
                        const int32_t* kv_len, const sv_paged_cache* cache);

/* Bytes of workspace that sv_kv_pages needs; 256 stands for none (the call then
 * takes a NULL workspace), 0 for sizes that the call would reject. */
size_t sv_kv_pages_workspace_size(int B, int T);

/* Pages of a cache for B requests: after the call request b holds the
 * ceil(kv_len[b] / page_size) pages that its length needs (a negative length
 * counts as 0), as the first entries of its page table's row.  All in place:
 *   page_table int32 [B, max_pages] with page_table_stride >= max_pages
 *              entries between rows.  Entries of pages given back become -1;
 *              those from pages_held[b] on are not read: initialise them to -1,
 *              so that no call sees tokens there.
 *   pages_held int32 [B], the pages that each request holds (counted as within
 *              0..max_pages).
 *   free_pages int32 [num_pages], free_count int32 [1]: the free pages are the
 *              first free_count[0] entries, a stack whose top is the last of
 *              them.
 *   shared_pages   int32 [B] or NULL (0): so many of the first pages that a
 *              request holds are not given back (others hold them too).
 * First pages are given back: the k-th of all (requests in order, a request's
 * pages in the order of its row) becomes the k-th from the top of the stack.
 * Then pages are taken: requests in order, each page from the top.  A request is
 * granted its pages if the stack has enough for all that the requests before it
 * and it itself lack; from the first that is not granted on, none is that lacks
 * a page, and what it holds stays as it was.  Nor is one that needs more than
 * max_pages.  Taking pages and giving the same ones back leaves the stack as it
 * was.
 *   granted    int32 [B] or NULL: 1 if the request holds what its length needs.
 *   query_start    int32 [B + 1] or NULL: packed new tokens, of which
 *   slots      int64 [T] or NULL gets page * page_size + place % page_size of
 *              each row's place, -1 where the request holds no page for it or
 *              the page is outside 0..num_pages-1, and
 *   positions  int64 [T] or NULL the place (as sv_rope and sv_qk_norm_rope take
 *              it); rows of no request are left as they were.
 *   page_size  a power of two up to SV_ATTN_MAX_PAGE.  num_pages, the pages of
 *              the cache, below 2^31; max_pages * page_size at most
 *              SV_ATTN_MAX_TOKENS.
 *   workspace  scratch of this call alone, 16-byte aligned.
 * A page should be held by one request only, but for shared ones, and not be
 * free as well; where it is not so no memory beyond the arrays is touched (what
 * is given back beyond num_pages entries is dropped). */
int sv_kv_pages(void* stream, int B, int T, int page_size, int max_pages, int num_pages, const int32_t* kv_len,
                const int32_t* shared_pages, const int32_t* query_start, int32_t* page_table,
                int64_t page_table_stride, int32_t* pages_held, int32_t* free_pages, int32_t* free_count,
                int32_t* granted, int64_t* slots, int64_t* positions, void* workspace, size_t workspace_bytes);

/* Reads tokens of a paged cache back into contiguous rows: row
 * row_start[b] + i of k_out and v_out, i < row_start[b+1] - row_start[b], gets
 * the token at place kv_begin[b] + i of request b (kv_begin NULL: 0), as the
 * value it stands for; zeros where the cache holds nothing.
 *   T          rows of the outputs; rows outside row_start[0] ..
 *              row_start[B] - 1 are left as they were.
 *   row_start  int32 [B + 1], ascending.
 *   out_dtype  SV_F32 or SV_BF16; k_out, v_out [T, cache->heads, head_dim]
 *              contiguous, 16-byte aligned.  Either may be NULL. */
int sv_kv_gather(void* stream, int B, int T, int out_dtype, const sv_paged_cache* cache, const int32_t* row_start,
                 const int32_t* kv_begin, void* k_out, void* v_out);

/* Bytes of workspace that sv_paged_attention needs for these sizes: 256 stands
 * for none (no context is split; the call then takes a NULL workspace), 0 for
 * sizes that the call would reject.  At most 2^29 + 1024. */
size_t sv_paged_attention_workspace_size(int B, int T, int q_heads, int kv_heads, int head_dim, int max_q_len,
                                         int max_kv_len);

/* Causal attention of the new tokens of B requests over their paged cache,
 * which already holds them.  Row r at place p of request b, head h: over the
 * tokens j of the request with j <= p (and j > p - window if window > 0),
 * whose key and value head is h / (q_heads / cache->heads),
 *   out = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale * (q . k_j)),
 *   lse = log(sum_j w_j)   (natural logarithm).
 * A row that sees no token gets out = 0 and lse = -infinity.  A token that a
 * row does not see has no influence on it, whatever its key and value hold.  A
 * NaN that a row sees shows: one in a key makes its whole result NaN, one in a
 * value the channel's at least.  An infinite value that a row sees makes the
 * channel's result infinite or NaN, and may make the row's others and its lse
 * NaN.
 * A score of -infinity (an infinite key) is a weight of zero, one of
 * +infinity makes its row NaN; a row whose weights are all zero gets what a row
 * that sees no token gets.  Scores are formed in binary32 and in base 2:
 * finite ones of 2.3e38 and more give no meaningful row.
 *   q, out     SV_BF16 elements, [T, q_heads, head_dim] with the given
 *              strides, 16-byte aligned, strides multiples of 8 elements (that
 *              of a dimension of one element is not looked at); no two of
 *              out's rows may overlap, nor out and q.  q_heads a multiple of
 *              cache->heads, T * q_heads below 2^31.
 *   lse        float [T, q_heads], or NULL.
 *   scale      > 0 and below 2.35e38 (usually head_dim^-0.5).
 *   max_q_len, max_kv_len   the most new tokens of a request and the largest
 *              kv_len, as far as the caller knows them (0: not known): they
 *              choose how the work is divided and change results by rounding
 *              only; larger requests are computed all the same.  Without
 *              max_q_len the average T / B is taken, and a request of more rows
 *              is worked off a tile after the other by the workgroups that an
 *              average one has: a prompt among decoding requests takes several
 *              times as long as with it.  Without max_kv_len no context is
 *              divided; a loose one costs workgroups and scratch.
 *   workspace  scratch of this call alone, 16-byte aligned; not a workspace of
 *              specverify.h's calls, whose cleared part it would overwrite.
 * Scores, sums and outputs are accumulated in binary32; the weights w_j are
 * rounded to bf16 for their product with the values (by up to 2^-8 of each; lse
 * and the sum that out is divided by have them unrounded). */
int sv_paged_attention(void* stream, int B, int T, int q_heads, const void* q, int64_t q_token_stride,
                       int64_t q_head_stride, const sv_paged_cache* cache, const int32_t* query_start,
                       const int32_t* kv_len, int max_q_len, int max_kv_len, float scale, int window, void* out,
                       int64_t out_token_stride, int64_t out_head_stride, float* lse, void* workspace,
                       size_t workspace_bytes);

/* Bytes of workspace that sv_paged_attention_sinks needs, as
 * sv_paged_attention_workspace_size. */
size_t sv_paged_attention_sinks_workspace_size(int B, int T, int q_heads, int kv_heads, int head_dim, int max_q_len,
                                               int max_kv_len, int window, int sinks);

/* sv_paged_attention with first tokens that stay visible beside the window: a
 * row at place p sees the tokens j <= p with j > p - window or j < sinks (all
 * j <= p with window 0).  Tokens between the two are not read, and the work is
 * divided by what a row sees rather than by max_kv_len.
 *   sinks      >= 0. */
int sv_paged_attention_sinks(void* stream, int B, int T, int q_heads, const void* q, int64_t q_token_stride,
                             int64_t q_head_stride, const sv_paged_cache* cache, const int32_t* query_start,
                             const int32_t* kv_len, int max_q_len, int max_kv_len, float scale, int window, int sinks,
                             void* out, int64_t out_token_stride, int64_t out_head_stride, float* lse, void* workspace,
                             size_t workspace_bytes);

/* Bytes of workspace that sv_paged_attention_shared needs (256: none); 0 for
 * sizes that the call would reject.  Every row has a part for each split of the
 * shared and of the own tokens, at least one of either: 4 (head_dim + 2) bytes a
 * part, token and query head. */
size_t sv_paged_attention_shared_workspace_size(int B, int T, int groups, int q_heads, int kv_heads, int head_dim,
                                                int max_q_len, int max_group_len, int max_shared_len, int max_own_len);

/* sv_paged_attention (without a window) for requests whose first tokens are the
 * same: group g is the requests group_start[g] .. group_start[g+1] - 1, whose
 * first shared_len[g] tokens are read once for all of them, through the page
 * table row of the first of them.  The rows of the others should hold the same
 * pages there, or copies (of a page that is shared in part, say): the result is
 * then that of sv_paged_attention but for roundings.  A row sees a shared token
 * j if j <= its place, as any other.
 *   groups     0: nothing is shared.
 *   group_start    int32 [groups + 1], ascending, within 0..B; requests outside
 *              group_start[0] .. group_start[groups] - 1 share nothing, nor do
 *              those of a group that reaches beyond the batch.
 *   shared_len     int32 [groups]; negative counts as 0.  The first request's row
 *              has to hold the shared pages also where that request has no rows,
 *              or a kv_len below shared_len.
 *   max_q_len, max_group_len, max_shared_len, max_own_len   the most new tokens
 *              of a request and of a group, the largest shared_len, and the
 *              largest number of tokens of a request that are not shared, as far
 *              as the caller knows them (0: not known; then contexts are not
 *              divided).  They choose how the work is divided, as in
 *              sv_paged_attention.
 * Worth it where the shared tokens are most of what a request's few rows read;
 * prompts of many rows, and requests with less in common than of their own, are
 * quicker with sv_paged_attention, which needs no part of every row either. */
int sv_paged_attention_shared(void* stream, int B, int T, int q_heads, const void* q, int64_t q_token_stride,
                              int64_t q_head_stride, const sv_paged_cache* cache, const int32_t* query_start,
                              const int32_t* kv_len, int groups, const int32_t* group_start, const int32_t* shared_len,
                              int max_q_len, int max_group_len, int max_shared_len, int max_own_len, float scale,
                              void* out, int64_t out_token_stride, int64_t out_head_stride, float* lse, void* workspace,
                              size_t workspace_bytes);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_ATTN_H */
