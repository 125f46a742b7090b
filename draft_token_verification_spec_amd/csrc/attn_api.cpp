// C entry points of specverify_attn.h: argument checks and launches on the
// caller's stream.  No call allocates, frees or synchronises the host.
#include <math.h>

#include "sv_attn.hpp"

using namespace sv;

namespace {

int to_status(hipError_t e) { return e == hipSuccess ? SV_OK : SV_ERR_HIP; }

bool rows_dtype_ok(int dtype) { return dtype == SV_F32 || dtype == SV_BF16; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Strides of rows [T, heads, D] that may be read, or that may be written (no
// two rows in one place).
bool read_strides_ok(int64_t token, int64_t head) { return token >= 0 && head >= 0; }
bool write_strides_ok(int T, int heads, int D, int64_t token, int64_t head) {
  return read_strides_ok(token, head) && (T <= 1 || token >= D) && (heads <= 1 || head >= D);
}

// Host checks of a cache; the tables and arrays may be missing where no call
// would read them (empty).
int check_cache(const sv_paged_cache* c, int B, bool empty) {
  if (!c) return SV_ERR_INVALID_ARG;
  if (c->dtype != SV_BF16 && c->dtype != SV_E4M3) return SV_ERR_INVALID_ARG;
  if (c->heads < 1 || c->head_dim < 16 || c->head_dim % 16 != 0 || c->page_size < 1 ||
      (c->page_size & (c->page_size - 1)) != 0 || c->num_pages < 0 || c->max_pages < 0)
    return SV_ERR_INVALID_ARG;
  if (c->heads > SV_ATTN_MAX_HEADS || c->head_dim > SV_ATTN_MAX_HEAD_DIM || c->page_size > SV_ATTN_MAX_PAGE ||
      int64_t(c->max_pages) * c->page_size > SV_ATTN_MAX_TOKENS)
    return SV_ERR_UNSUPPORTED;
  if (empty) return SV_OK;
  if (c->page_table_stride < 0 || (c->page_table_stride < c->max_pages && c->page_table_stride != 0 && B > 1))
    return SV_ERR_INVALID_ARG;
  if (c->max_pages > 0 && !c->page_table) return SV_ERR_INVALID_ARG;
  const int64_t unit = c->dtype == SV_BF16 ? 8 : 16;  // elements of 16 bytes
  for (int64_t s : {c->k_page_stride, c->k_token_stride, c->k_head_stride, c->v_page_stride, c->v_token_stride,
                    c->v_head_stride})
    if (s < 0 || s % unit != 0 || s / unit > int64_t(0xffffffffu)) return SV_ERR_INVALID_ARG;
  for (int64_t s : {c->k_page_stride, c->v_page_stride})
    if (c->num_pages > 1 && s < c->head_dim) return SV_ERR_INVALID_ARG;
  if (!write_strides_ok(c->page_size, c->heads, c->head_dim, c->k_token_stride, c->k_head_stride) ||
      !write_strides_ok(c->page_size, c->heads, c->head_dim, c->v_token_stride, c->v_head_stride))
    return SV_ERR_INVALID_ARG;
  if (!aligned16(c->k) || !aligned16(c->v)) return SV_ERR_INVALID_ARG;
  if (c->num_pages > 0 && (!c->k || !c->v)) return SV_ERR_INVALID_ARG;
  if (c->num_pages > 0 && c->dtype == SV_E4M3 && (!c->k_scale || !c->v_scale)) return SV_ERR_INVALID_ARG;
  return SV_OK;
}

PagedView view_of(const sv_paged_cache* c) {
  PagedView v;
  v.table = c->page_table;
  v.table_stride = c->page_table_stride;
  v.max_pages = c->num_pages > 0 ? c->max_pages : 0;  // a cache without pages holds nothing
  v.num_pages = c->num_pages;
  v.heads = c->heads;
  v.D = c->head_dim;
  v.page_shift = __builtin_ctz(unsigned(c->page_size));
  v.k = c->k;
  v.v = c->v;
  v.k_page = c->k_page_stride;
  v.k_token = c->k_token_stride;
  v.k_head = c->k_head_stride;
  v.v_page = c->v_page_stride;
  v.v_token = c->v_token_stride;
  v.v_head = c->v_head_stride;
  v.k_scale = c->k_scale;
  v.v_scale = c->v_scale;
  return v;
}

int check_batch(int B, int T) {
  if (B < 0 || T < 0) return SV_ERR_INVALID_ARG;
  if (B > SV_MAX_B || T > SV_ATTN_MAX_ROWS) return SV_ERR_UNSUPPORTED;
  return SV_OK;
}

int check_attention_sizes(int B, int T, int q_heads, int kv_heads, int head_dim, int max_q_len, int max_kv_len) {
  const int st = check_batch(B, T);
  if (st != SV_OK) return st;
  if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || head_dim < 16 || head_dim % 16 != 0 ||
      max_q_len < 0 || max_kv_len < 0)
    return SV_ERR_INVALID_ARG;
  if (q_heads > SV_ATTN_MAX_HEADS || head_dim > SV_ATTN_MAX_HEAD_DIM || int64_t(T) * q_heads > INT32_MAX)
    return SV_ERR_UNSUPPORTED;  // (a request's rows times heads are counted in 32 bits)
  return SV_OK;
}

// A norm's arguments; rows are checked by row_strides_ok.
bool norm_ok(int weight_dtype, float eps) {
  return rows_dtype_ok(weight_dtype) && eps >= 1.17549435e-38f && isfinite(eps);
}

int append(void* stream, int B, int T, int q_heads, int dtype, int rotary_dim, int layout, const double* freq,
           float mscale, const int64_t* positions, const NormWeights* norm, const RowsIn& q, const RowsOut& q_out,
           const RowsIn& k, const RowsIn& v, const int32_t* query_start, const int32_t* kv_len,
           const sv_paged_cache* cache) {
  int st = check_batch(B, T);
  if (st != SV_OK) return st;
  const bool empty = B == 0 || T == 0;
  st = check_cache(cache, B, empty);
  if (st != SV_OK) return st;
  if (q_heads < 0 || !rows_dtype_ok(dtype) || rotary_dim < 0 || rotary_dim % 2 != 0 || rotary_dim > cache->head_dim ||
      (layout != SV_ROPE_HALF && layout != SV_ROPE_INTERLEAVED) || !isfinite(mscale) ||
      (norm && !norm_ok(norm->dtype, norm->eps)))
    return SV_ERR_INVALID_ARG;
  if (q_heads > SV_ATTN_MAX_HEADS) return SV_ERR_UNSUPPORTED;
  if (empty) return SV_OK;
  if (!k.p || !v.p || !query_start || !kv_len || (rotary_dim > 0 && !freq) || (q_heads > 0 && (!q.p || !q_out.p)))
    return SV_ERR_INVALID_ARG;
  if (!read_strides_ok(k.token, k.head) || !read_strides_ok(v.token, v.head)) return SV_ERR_INVALID_ARG;
  if (q_heads > 0 && (!read_strides_ok(q.token, q.head) ||
                      !write_strides_ok(T, q_heads, cache->head_dim, q_out.token, q_out.head)))
    return SV_ERR_INVALID_ARG;
  AppendArgs a;
  a.B = B;
  a.T = T;
  a.q_heads = q_heads;
  a.rotary = rotary_dim;
  a.layout = layout;
  a.freq = freq;
  a.mscale = mscale;
  a.positions = positions;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = q_out;
  a.query_start = query_start;
  a.kv_len = kv_len;
  a.cache = view_of(cache);
  if (norm) a.norm = *norm;
  return to_status((norm ? launch_append_normed : launch_append)(a, dtype, cache->dtype, static_cast<hipStream_t>(stream)));
}

// Sizes, types and pointers of sv_qk_norm_rope and its backward pass;
// SV_OK with a.T set to 0 if there is nothing to do.
int check_norm(NormRopeArgs& a, int dtype, bool backward) {
  if (a.T < 0 || a.q_heads < 0 || a.k_heads < 0 || a.D < 1 || a.rotary < 0 || a.rotary % 2 != 0 || a.rotary > a.D ||
      !rows_dtype_ok(dtype) || (a.layout != SV_ROPE_HALF && a.layout != SV_ROPE_INTERLEAVED) || !isfinite(a.mscale) ||
      !norm_ok(a.norm.dtype, a.norm.eps))
    return SV_ERR_INVALID_ARG;
  if (a.D > SV_ATTN_MAX_HEAD_DIM || a.q_heads > SV_ATTN_MAX_HEADS || a.k_heads > SV_ATTN_MAX_HEADS ||
      a.T > SV_ATTN_MAX_ROWS)
    return SV_ERR_UNSUPPORTED;
  if (a.q_heads == 0 && a.k_heads == 0) a.T = 0;
  if (a.T == 0) return SV_OK;
  if (a.rotary > 0 && (!a.freq || !a.positions)) return SV_ERR_INVALID_ARG;
  auto rows_ok = [&](int heads, const RowsIn& x, const RowsIn& grad, const RowsOut& out) {
    return heads == 0 || (x.p && out.p && read_strides_ok(x.token, x.head) &&
                          write_strides_ok(a.T, heads, a.D, out.token, out.head) &&
                          (!backward || (grad.p && read_strides_ok(grad.token, grad.head))));
  };
  return rows_ok(a.q_heads, a.q, a.dq, a.q_out) && rows_ok(a.k_heads, a.k, a.dk, a.k_out) ? SV_OK : SV_ERR_INVALID_ARG;
}

size_t norm_scratch(int T, int D) { return size_t(norm_parts(T)) * 2 * D * sizeof(float); }

// Checks of an attention call, and its arguments where there is something to do
// (a.T is 0 otherwise).  The plan and the parts are the caller's part.
int check_attention(AttnArgs& a, int B, int T, int q_heads, const RowsIn& q, const sv_paged_cache* cache,
                    const int32_t* query_start, const int32_t* kv_len, int max_q_len, int max_kv_len, float scale,
                    int window, const RowsOut& out, float* lse) {
  a.T = 0;
  int st = check_batch(B, T);
  if (st != SV_OK) return st;
  const bool empty = B == 0 || T == 0;
  st = check_cache(cache, B, empty);
  if (st != SV_OK) return st;
  st = check_attention_sizes(B, T, q_heads, cache->heads, cache->head_dim, max_q_len, max_kv_len);
  if (st != SV_OK) return st;
  if (!(scale > 0.f) || !isfinite(scale * 1.4426950408889634f) || window < 0) return SV_ERR_INVALID_ARG;
  if (empty) return SV_OK;
  if (!q.p || !out.p || !query_start || !kv_len || !aligned16(q.p) || !aligned16(out.p)) return SV_ERR_INVALID_ARG;
  for (int64_t s : {q.token, out.token})
    if (s < 0 || (T > 1 && s % 8 != 0)) return SV_ERR_INVALID_ARG;
  for (int64_t s : {q.head, out.head})
    if (s < 0 || (q_heads > 1 && s % 8 != 0)) return SV_ERR_INVALID_ARG;
  if (!write_strides_ok(T, q_heads, cache->head_dim, out.token, out.head)) return SV_ERR_INVALID_ARG;
  a.B = B;
  a.T = T;
  a.q_heads = q_heads;
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.query_start = query_start;
  a.kv_len = kv_len;
  a.scale = scale;
  a.window = window;
  a.sinks = 0;
  a.groups = 0;
  a.group_start = a.shared_len = nullptr;
  const PagedView v = view_of(cache);
  const int shift = cache->dtype == SV_BF16 ? 3 : 4;  // elements of 16 bytes
  a.cache.table = v.table;
  a.cache.table_stride = v.table_stride;
  a.cache.k = v.k;
  a.cache.v = v.v;
  a.cache.k_scale = v.k_scale;
  a.cache.v_scale = v.v_scale;
  a.cache.ku = {uint32_t(v.k_page >> shift), uint32_t(v.k_token >> shift), uint32_t(v.k_head >> shift)};
  a.cache.vu = {uint32_t(v.v_page >> shift), uint32_t(v.v_token >> shift), uint32_t(v.v_head >> shift)};
  a.cache.max_pages = v.max_pages;
  a.cache.num_pages = v.num_pages;
  a.cache.heads = v.heads;
  a.cache.D = v.D;
  a.cache.page_shift = v.page_shift;
  return SV_OK;
}

bool scratch_ok(const void* workspace, size_t have, size_t need) {
  return need == 0 || (workspace && aligned16(workspace) && have >= 256 + need);
}

// A plan's parts in the workspace.
void place_parts(AttnPlan& p, void* workspace) {
  p.part_ml = static_cast<float2*>(workspace);
  p.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.ml_bytes);
}

}  // namespace

extern "C" {

int sv_rope_frequencies(int rotary_dim, double base, int scaling, double factor, double original_len, double low,
                        double high, double* freq, float* mscale) {
  if (rotary_dim < 0 || rotary_dim % 2 != 0 || !(base > 0) || !isfinite(base) || !mscale || (rotary_dim > 0 && !freq))
    return SV_ERR_INVALID_ARG;
  if (scaling < SV_ROPE_PLAIN || scaling > SV_ROPE_BANDS) return SV_ERR_INVALID_ARG;
  if (scaling != SV_ROPE_PLAIN && !(factor >= 1.0 && isfinite(factor))) return SV_ERR_INVALID_ARG;
  const bool ramped = scaling == SV_ROPE_RAMP || scaling == SV_ROPE_BANDS;
  if (ramped && !(original_len > 0 && isfinite(original_len) && low > 0 && low < high && isfinite(high)))
    return SV_ERR_INVALID_ARG;
  if (scaling == SV_ROPE_RAMP && !(base > 1.0)) return SV_ERR_INVALID_ARG;  // pairs have to turn ever slower
  if (scaling == SV_ROPE_BASE && rotary_dim <= 2) return SV_ERR_INVALID_ARG;
  const double d = rotary_dim, pi2 = 6.283185307179586477;
  if (scaling == SV_ROPE_BASE) base *= pow(factor, d / (d - 2));
  // the (real-valued) pair index whose frequency turns n times over original_len
  auto pair_turning = [&](double n) { return d * log(original_len / (n * pi2)) / (2 * log(base)); };
  double first = 0, last = 0;
  if (scaling == SV_ROPE_RAMP) {
    first = fmax(floor(pair_turning(high)), 0.0);
    last = fmin(ceil(pair_turning(low)), d - 1);
    if (last <= first) last = first + 0.001;
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double f = pow(base, -2.0 * i / d);
    double kept = 1;  // the share of f that is not divided by factor
    if (scaling == SV_ROPE_LINEAR) kept = 0;
    if (scaling == SV_ROPE_RAMP) kept = 1 - fmin(fmax((i - first) / (last - first), 0.0), 1.0);
    if (scaling == SV_ROPE_BANDS) kept = fmin(fmax((original_len * f / pi2 - low) / (high - low), 0.0), 1.0);
    freq[i] = scaling == SV_ROPE_PLAIN || scaling == SV_ROPE_BASE ? f : kept * f + (1 - kept) * (f / factor);
  }
  *mscale = scaling == SV_ROPE_RAMP ? float(0.1 * log(factor) + 1.0) : 1.f;
  return SV_OK;
}

int sv_rope(void* stream, int T, int heads, int head_dim, int rotary_dim, int layout, int backward, int dtype,
            const void* x, int64_t x_token_stride, int64_t x_head_stride, const int64_t* positions,
            const double* freq, float mscale, void* out, int64_t out_token_stride, int64_t out_head_stride) {
  if (T < 0 || heads < 0 || head_dim < 1 || rotary_dim < 0 || rotary_dim % 2 != 0 || rotary_dim > head_dim ||
      !rows_dtype_ok(dtype) || (layout != SV_ROPE_HALF && layout != SV_ROPE_INTERLEAVED) || !isfinite(mscale))
    return SV_ERR_INVALID_ARG;
  if (head_dim > SV_ATTN_MAX_HEAD_DIM || heads > SV_ATTN_MAX_HEADS || T > SV_ATTN_MAX_ROWS)
    return SV_ERR_UNSUPPORTED;
  if (T == 0 || heads == 0) return SV_OK;
  if (!x || !out || !positions || (rotary_dim > 0 && !freq)) return SV_ERR_INVALID_ARG;
  if (!read_strides_ok(x_token_stride, x_head_stride) ||
      !write_strides_ok(T, heads, head_dim, out_token_stride, out_head_stride))
    return SV_ERR_INVALID_ARG;
  RopeArgs a;
  a.T = T;
  a.heads = heads;
  a.D = head_dim;
  a.rotary = rotary_dim;
  a.layout = layout;
  a.backward = backward ? 1 : 0;
  a.x = {x, x_token_stride, x_head_stride};
  a.out = {out, out_token_stride, out_head_stride};
  a.positions = positions;
  a.freq = freq;
  a.mscale = mscale;
  return to_status(launch_rope(a, dtype, static_cast<hipStream_t>(stream)));
}

int sv_kv_append(void* stream, int B, int T, int q_heads, int dtype, int rotary_dim, int layout, const double* freq,
                 float mscale, const int64_t* positions, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                 void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride, const void* k,
                 int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
                 int64_t v_head_stride, const int32_t* query_start, const int32_t* kv_len,
                 const sv_paged_cache* cache) {
  return append(stream, B, T, q_heads, dtype, rotary_dim, layout, freq, mscale, positions, nullptr,
                {q, q_token_stride, q_head_stride}, {q_out, q_out_token_stride, q_out_head_stride},
                {k, k_token_stride, k_head_stride}, {v, v_token_stride, v_head_stride}, query_start, kv_len, cache);
}

int sv_kv_append_normed(void* stream, int B, int T, int q_heads, int dtype, int rotary_dim, int layout,
                        const double* freq, float mscale, const int64_t* positions, int weight_dtype,
                        const void* q_weight, const void* k_weight, float eps, const void* q, int64_t q_token_stride,
                        int64_t q_head_stride, void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                        const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                        int64_t v_token_stride, int64_t v_head_stride, const int32_t* query_start,
                        const int32_t* kv_len, const sv_paged_cache* cache) {
  NormWeights norm = {q_weight, k_weight, weight_dtype, eps, 0.};
  if (cache && cache->head_dim > 0) norm.inv_dim = 1. / cache->head_dim;
  return append(stream, B, T, q_heads, dtype, rotary_dim, layout, freq, mscale, positions, &norm,
                {q, q_token_stride, q_head_stride}, {q_out, q_out_token_stride, q_out_head_stride},
                {k, k_token_stride, k_head_stride}, {v, v_token_stride, v_head_stride}, query_start, kv_len, cache);
}

int sv_qk_norm_rope(void* stream, int T, int q_heads, int k_heads, int head_dim, int rotary_dim, int layout, int dtype,
                    const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
                    int64_t k_token_stride, int64_t k_head_stride, int weight_dtype, const void* q_weight,
                    const void* k_weight, float eps, const int64_t* positions, const double* freq, float mscale,
                    void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride, void* k_out,
                    int64_t k_out_token_stride, int64_t k_out_head_stride) {
  NormRopeArgs a = {T, q_heads, k_heads, head_dim, rotary_dim, layout, {q_weight, k_weight, weight_dtype, eps, 1. / head_dim}};
  a.q = {q, q_token_stride, q_head_stride};
  a.k = {k, k_token_stride, k_head_stride};
  a.q_out = {q_out, q_out_token_stride, q_out_head_stride};
  a.k_out = {k_out, k_out_token_stride, k_out_head_stride};
  a.positions = positions;
  a.freq = freq;
  a.mscale = mscale;
  const int st = check_norm(a, dtype, false);
  if (st != SV_OK || a.T == 0) return st;
  return to_status(launch_norm(a, dtype, static_cast<hipStream_t>(stream)));
}

size_t sv_qk_norm_rope_backward_workspace_size(int T, int head_dim) {
  if (T < 0 || T > SV_ATTN_MAX_ROWS || head_dim < 1 || head_dim > SV_ATTN_MAX_HEAD_DIM) return 0;
  return 256 + norm_scratch(T, head_dim);
}

int sv_qk_norm_rope_backward(void* stream, int T, int q_heads, int k_heads, int head_dim, int rotary_dim, int layout,
                             int dtype, const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
                             int64_t k_token_stride, int64_t k_head_stride, const void* dq_out,
                             int64_t dq_out_token_stride, int64_t dq_out_head_stride, const void* dk_out,
                             int64_t dk_out_token_stride, int64_t dk_out_head_stride, int weight_dtype,
                             const void* q_weight, const void* k_weight, float eps, const int64_t* positions,
                             const double* freq, float mscale, void* dq, int64_t dq_token_stride,
                             int64_t dq_head_stride, void* dk, int64_t dk_token_stride, int64_t dk_head_stride,
                             float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes) {
  NormRopeArgs a = {T, q_heads, k_heads, head_dim, rotary_dim, layout, {q_weight, k_weight, weight_dtype, eps, 1. / head_dim}};
  a.q = {q, q_token_stride, q_head_stride};
  a.k = {k, k_token_stride, k_head_stride};
  a.dq = {dq_out, dq_out_token_stride, dq_out_head_stride};
  a.dk = {dk_out, dk_out_token_stride, dk_out_head_stride};
  a.q_out = {dq, dq_token_stride, dq_head_stride};
  a.k_out = {dk, dk_token_stride, dk_head_stride};
  a.positions = positions;
  a.freq = freq;
  a.mscale = mscale;
  a.dq_weight = dq_weight;
  a.dk_weight = dk_weight;
  const int st = check_norm(a, dtype, true);
  if (st != SV_OK) return st;
  const bool weights = dq_weight || dk_weight;
  if (a.T == 0 && !weights) return SV_OK;
  if (weights && a.T > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < 256 + norm_scratch(T, head_dim)))
    return SV_ERR_WORKSPACE;
  a.part = weights ? static_cast<float*>(workspace) : nullptr;
  return to_status(launch_norm_backward(a, dtype, static_cast<hipStream_t>(stream)));
}

size_t sv_kv_pages_workspace_size(int B, int T) {
  return check_batch(B, T) == SV_OK ? 256 + pages_scratch(B, T) : 0;
}

int sv_kv_pages(void* stream, int B, int T, int page_size, int max_pages, int num_pages, const int32_t* kv_len,
                const int32_t* shared_pages, const int32_t* query_start, int32_t* page_table,
                int64_t page_table_stride, int32_t* pages_held, int32_t* free_pages, int32_t* free_count,
                int32_t* granted, int64_t* slots, int64_t* positions, void* workspace, size_t workspace_bytes) {
  const int st = check_batch(B, T);
  if (st != SV_OK) return st;
  if (page_size < 1 || (page_size & (page_size - 1)) != 0 || max_pages < 0 || num_pages < 0) return SV_ERR_INVALID_ARG;
  if (page_size > SV_ATTN_MAX_PAGE || int64_t(max_pages) * page_size > SV_ATTN_MAX_TOKENS) return SV_ERR_UNSUPPORTED;
  if (B == 0) return SV_OK;
  if (!kv_len || !pages_held || !free_count || (max_pages > 0 && !page_table) || (num_pages > 0 && !free_pages) ||
      (B > 1 && page_table_stride < max_pages) || page_table_stride < 0 || ((slots || positions) && T > 0 && !query_start))
    return SV_ERR_INVALID_ARG;
  if (!slots && !positions) query_start = nullptr;
  if (pages_scratch(B, T) != 0 &&
      (!workspace || !aligned16(workspace) || workspace_bytes < 256 + pages_scratch(B, T)))
    return SV_ERR_WORKSPACE;
  PagesArgs a;
  a.B = B;
  a.T = T;
  a.page_shift = __builtin_ctz(unsigned(page_size));
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.kv_len = kv_len;
  a.shared = shared_pages;
  a.query_start = T > 0 ? query_start : nullptr;
  a.table = page_table;
  a.table_stride = page_table_stride;
  a.held = pages_held;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.granted = granted;
  a.slots = slots;
  a.positions = positions;
  a.scratch = workspace;
  return to_status(launch_pages(a, static_cast<hipStream_t>(stream)));
}

int sv_kv_gather(void* stream, int B, int T, int out_dtype, const sv_paged_cache* cache, const int32_t* row_start,
                 const int32_t* kv_begin, void* k_out, void* v_out) {
  int st = check_batch(B, T);
  if (st != SV_OK) return st;
  const bool empty = B == 0 || T == 0 || (!k_out && !v_out);
  st = check_cache(cache, B, empty);
  if (st != SV_OK) return st;
  if (!rows_dtype_ok(out_dtype)) return SV_ERR_INVALID_ARG;
  if (empty) return SV_OK;
  if (!row_start || !aligned16(k_out) || !aligned16(v_out)) return SV_ERR_INVALID_ARG;
  GatherArgs a;
  a.B = B;
  a.T = T;
  a.row_start = row_start;
  a.kv_begin = kv_begin;
  a.k_out = k_out;
  a.v_out = v_out;
  a.cache = view_of(cache);
  return to_status(launch_gather(a, out_dtype, cache->dtype, static_cast<hipStream_t>(stream)));
}

size_t sv_paged_attention_workspace_size(int B, int T, int q_heads, int kv_heads, int head_dim, int max_q_len,
                                         int max_kv_len) {
  if (check_attention_sizes(B, T, q_heads, kv_heads, head_dim, max_q_len, max_kv_len) != SV_OK) return 0;
  const AttnPlan p = plan_attention(B, T, q_heads, kv_heads, head_dim, max_q_len, max_kv_len);
  return 256 + p.ml_bytes + p.o_bytes;
}

int sv_paged_attention(void* stream, int B, int T, int q_heads, const void* q, int64_t q_token_stride,
                       int64_t q_head_stride, const sv_paged_cache* cache, const int32_t* query_start,
                       const int32_t* kv_len, int max_q_len, int max_kv_len, float scale, int window, void* out,
                       int64_t out_token_stride, int64_t out_head_stride, float* lse, void* workspace,
                       size_t workspace_bytes) {
  AttnArgs a;
  const int st = check_attention(a, B, T, q_heads, {q, q_token_stride, q_head_stride}, cache, query_start, kv_len,
                                 max_q_len, max_kv_len, scale, window, {out, out_token_stride, out_head_stride}, lse);
  if (st != SV_OK || a.T == 0) return st;
  AttnPlan p = plan_attention(B, T, q_heads, cache->heads, cache->head_dim, max_q_len, max_kv_len);
  if (!scratch_ok(workspace, workspace_bytes, p.ml_bytes + p.o_bytes)) return SV_ERR_WORKSPACE;
  place_parts(p, workspace);
  return to_status(launch_attention(a, p, cache->dtype, static_cast<hipStream_t>(stream)));
}

size_t sv_paged_attention_sinks_workspace_size(int B, int T, int q_heads, int kv_heads, int head_dim, int max_q_len,
                                               int max_kv_len, int window, int sinks) {
  if (check_attention_sizes(B, T, q_heads, kv_heads, head_dim, max_q_len, max_kv_len) != SV_OK || window < 0 || sinks < 0)
    return 0;
  const AttnPlan p = plan_sinks(B, T, q_heads, kv_heads, head_dim, max_q_len, max_kv_len, window, sinks);
  return 256 + p.ml_bytes + p.o_bytes;
}

int sv_paged_attention_sinks(void* stream, int B, int T, int q_heads, const void* q, int64_t q_token_stride,
                             int64_t q_head_stride, const sv_paged_cache* cache, const int32_t* query_start,
                             const int32_t* kv_len, int max_q_len, int max_kv_len, float scale, int window, int sinks,
                             void* out, int64_t out_token_stride, int64_t out_head_stride, float* lse, void* workspace,
                             size_t workspace_bytes) {
  AttnArgs a;
  const int st = check_attention(a, B, T, q_heads, {q, q_token_stride, q_head_stride}, cache, query_start, kv_len,
                                 max_q_len, max_kv_len, scale, window, {out, out_token_stride, out_head_stride}, lse);
  if (st != SV_OK) return st;
  if (sinks < 0) return SV_ERR_INVALID_ARG;
  if (a.T == 0) return SV_OK;
  a.sinks = sinks;
  AttnPlan p = plan_sinks(B, T, q_heads, cache->heads, cache->head_dim, max_q_len, max_kv_len, window, sinks);
  if (!scratch_ok(workspace, workspace_bytes, p.ml_bytes + p.o_bytes)) return SV_ERR_WORKSPACE;
  place_parts(p, workspace);
  return to_status(launch_sinks(a, p, cache->dtype, static_cast<hipStream_t>(stream)));
}

size_t sv_paged_attention_shared_workspace_size(int B, int T, int groups, int q_heads, int kv_heads, int head_dim,
                                                int max_q_len, int max_group_len, int max_shared_len, int max_own_len) {
  if (check_attention_sizes(B, T, q_heads, kv_heads, head_dim, max_q_len, max_own_len) != SV_OK || groups < 0 ||
      groups > SV_MAX_B || max_group_len < 0 || max_shared_len < 0)
    return 0;
  if (groups == 0) return sv_paged_attention_workspace_size(B, T, q_heads, kv_heads, head_dim, max_q_len, max_own_len);
  return 256 + plan_shared(B, T, groups, q_heads, kv_heads, head_dim, max_q_len, max_group_len, max_shared_len,
                           max_own_len).bytes;
}

int sv_paged_attention_shared(void* stream, int B, int T, int q_heads, const void* q, int64_t q_token_stride,
                              int64_t q_head_stride, const sv_paged_cache* cache, const int32_t* query_start,
                              const int32_t* kv_len, int groups, const int32_t* group_start, const int32_t* shared_len,
                              int max_q_len, int max_group_len, int max_shared_len, int max_own_len, float scale,
                              void* out, int64_t out_token_stride, int64_t out_head_stride, float* lse, void* workspace,
                              size_t workspace_bytes) {
  if (groups == 0)  // nothing is shared
    return sv_paged_attention(stream, B, T, q_heads, q, q_token_stride, q_head_stride, cache, query_start, kv_len,
                              max_q_len, max_own_len, scale, 0, out, out_token_stride, out_head_stride, lse, workspace,
                              workspace_bytes);
  AttnArgs a;
  const int st = check_attention(a, B, T, q_heads, {q, q_token_stride, q_head_stride}, cache, query_start, kv_len,
                                 max_q_len, max_own_len, scale, 0, {out, out_token_stride, out_head_stride}, lse);
  if (st != SV_OK) return st;
  if (groups < 0 || max_group_len < 0 || max_shared_len < 0) return SV_ERR_INVALID_ARG;
  if (groups > SV_MAX_B) return SV_ERR_UNSUPPORTED;
  if (a.T == 0) return SV_OK;
  if (!group_start || !shared_len) return SV_ERR_INVALID_ARG;
  a.groups = groups;
  a.group_start = group_start;
  a.shared_len = shared_len;
  SharedPlan p = plan_shared(B, T, groups, q_heads, cache->heads, cache->head_dim, max_q_len, max_group_len,
                             max_shared_len, max_own_len);
  if (!scratch_ok(workspace, workspace_bytes, p.bytes)) return SV_ERR_WORKSPACE;
  place_parts(p.shared, workspace);
  place_parts(p.own, workspace);
  return to_status(launch_shared(a, p, cache->dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
