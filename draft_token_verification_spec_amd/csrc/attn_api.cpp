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
  int st = check_batch(B, T);
  if (st != SV_OK) return st;
  const bool empty = B == 0 || T == 0;
  st = check_cache(cache, B, empty);
  if (st != SV_OK) return st;
  if (q_heads < 0 || !rows_dtype_ok(dtype) || rotary_dim < 0 || rotary_dim % 2 != 0 || rotary_dim > cache->head_dim ||
      (layout != SV_ROPE_HALF && layout != SV_ROPE_INTERLEAVED) || !isfinite(mscale))
    return SV_ERR_INVALID_ARG;
  if (q_heads > SV_ATTN_MAX_HEADS) return SV_ERR_UNSUPPORTED;
  if (empty) return SV_OK;
  if (!k || !v || !query_start || !kv_len || (rotary_dim > 0 && !freq) || (q_heads > 0 && (!q || !q_out)))
    return SV_ERR_INVALID_ARG;
  if (!read_strides_ok(k_token_stride, k_head_stride) || !read_strides_ok(v_token_stride, v_head_stride))
    return SV_ERR_INVALID_ARG;
  if (q_heads > 0 && (!read_strides_ok(q_token_stride, q_head_stride) ||
                      !write_strides_ok(T, q_heads, cache->head_dim, q_out_token_stride, q_out_head_stride)))
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
  a.q = {q, q_token_stride, q_head_stride};
  a.k = {k, k_token_stride, k_head_stride};
  a.v = {v, v_token_stride, v_head_stride};
  a.q_out = {q_out, q_out_token_stride, q_out_head_stride};
  a.query_start = query_start;
  a.kv_len = kv_len;
  a.cache = view_of(cache);
  return to_status(launch_append(a, dtype, cache->dtype, static_cast<hipStream_t>(stream)));
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
  int st = check_batch(B, T);
  if (st != SV_OK) return st;
  const bool empty = B == 0 || T == 0;
  st = check_cache(cache, B, empty);
  if (st != SV_OK) return st;
  st = check_attention_sizes(B, T, q_heads, cache->heads, cache->head_dim, max_q_len, max_kv_len);
  if (st != SV_OK) return st;
  if (!(scale > 0.f) || !isfinite(scale * 1.4426950408889634f) || window < 0) return SV_ERR_INVALID_ARG;
  if (empty) return SV_OK;
  if (!q || !out || !query_start || !kv_len || !aligned16(q) || !aligned16(out)) return SV_ERR_INVALID_ARG;
  for (int64_t s : {q_token_stride, out_token_stride})
    if (s < 0 || (T > 1 && s % 8 != 0)) return SV_ERR_INVALID_ARG;
  for (int64_t s : {q_head_stride, out_head_stride})
    if (s < 0 || (q_heads > 1 && s % 8 != 0)) return SV_ERR_INVALID_ARG;
  if (!write_strides_ok(T, q_heads, cache->head_dim, out_token_stride, out_head_stride)) return SV_ERR_INVALID_ARG;
  AttnPlan p = plan_attention(B, T, q_heads, cache->heads, cache->head_dim, max_q_len, max_kv_len);
  if (p.num_splits > 1 &&
      (!workspace || !aligned16(workspace) || workspace_bytes < 256 + p.ml_bytes + p.o_bytes))
    return SV_ERR_WORKSPACE;
  p.part_ml = static_cast<float2*>(workspace);
  p.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.ml_bytes);
  AttnArgs a;
  a.B = B;
  a.T = T;
  a.q_heads = q_heads;
  a.q = {q, q_token_stride, q_head_stride};
  a.out = {out, out_token_stride, out_head_stride};
  a.lse = lse;
  a.query_start = query_start;
  a.kv_len = kv_len;
  a.scale = scale;
  a.window = window;
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
  return to_status(launch_attention(a, p, cache->dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
