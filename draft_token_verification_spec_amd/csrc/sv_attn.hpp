// Launchers of the rotary, cache and attention kernels (attn_api.cpp checks
// the arguments).
#pragma once

#include "sv_paged.hpp"

namespace sv {

// Rows x [T, heads, D] with strides between rows and heads, in elements.
struct RowsIn {
  const void* p;
  int64_t token, head;
};
struct RowsOut {
  void* p;
  int64_t token, head;
};

struct RopeArgs {
  int T, heads, D, rotary;
  int layout, backward;
  RowsIn x;
  RowsOut out;
  const int64_t* positions;
  const double* freq;
  float mscale;
};
hipError_t launch_rope(const RopeArgs& a, int dtype, hipStream_t stream);

// Norms of query and key heads: weights of head_dim channels (null: ones).
struct NormWeights {
  const void* q;
  const void* k;
  int dtype;
  float eps;
  double inv_dim;  // 1 / head_dim
};

// Queries and keys [T, heads, D] normed and turned, or (launch_norm_backward)
// the gradients of that: dq, dk with respect to its outputs come in, q_out,
// k_out with respect to q, k and the weights' go out.
struct NormRopeArgs {
  int T, q_heads, k_heads, D, rotary;
  int layout;
  NormWeights norm;
  RowsIn q, k, dq, dk;
  RowsOut q_out, k_out;
  const int64_t* positions;
  const double* freq;
  float mscale;
  float* part;       // [norm_parts(T)][2][D], the weights' gradients of a workgroup's rows
  float* dq_weight;  // nullable
  float* dk_weight;  // nullable
};
int norm_parts(int T);  // workgroups of the backward pass
hipError_t launch_norm(const NormRopeArgs& a, int dtype, hipStream_t stream);
hipError_t launch_norm_backward(const NormRopeArgs& a, int dtype, hipStream_t stream);

struct AppendArgs {
  int B, T, q_heads, rotary;
  int layout;
  const double* freq;
  float mscale;
  const int64_t* positions;  // nullable
  RowsIn q, k, v;
  RowsOut q_out;
  const int32_t* query_start;
  const int32_t* kv_len;
  PagedView cache;
  NormWeights norm;  // launch_append_normed
};
hipError_t launch_append(const AppendArgs& a, int dtype, int cache_dtype, hipStream_t stream);
hipError_t launch_append_normed(const AppendArgs& a, int dtype, int cache_dtype, hipStream_t stream);

// Pages taken and given back.  scratch: pages_scratch(B, T) bytes (0: none).
struct PagesArgs {
  int B, T;
  int page_shift, max_pages, num_pages;
  const int32_t* kv_len;
  const int32_t* shared;       // nullable
  const int32_t* query_start;  // nullable: no rows
  int32_t* table;
  int64_t table_stride;
  int32_t* held;
  int32_t* free_pages;
  int32_t* free_count;
  int32_t* granted;    // nullable
  int64_t* slots;      // nullable
  int64_t* positions;  // nullable
  void* scratch;
};
size_t pages_scratch(int B, int T);
hipError_t launch_pages(const PagesArgs& a, hipStream_t stream);

struct GatherArgs {
  int B, T;
  const int32_t* row_start;
  const int32_t* kv_begin;  // nullable
  void* k_out;              // nullable
  void* v_out;              // nullable
  PagedView cache;
};
hipError_t launch_gather(const GatherArgs& a, int out_dtype, int cache_dtype, hipStream_t stream);

// Strides in units of 16 bytes.
struct UnitStrides {
  uint32_t page, token, head;
};

// A cache as the attention reads it.
struct CacheView {
  const int32_t* table;
  int64_t table_stride;
  const void* k;
  const void* v;
  const uint8_t* k_scale;
  const uint8_t* v_scale;
  UnitStrides ku, vu;
  int max_pages, num_pages, heads, D, page_shift;
};

struct AttnArgs {
  int B, T, q_heads;
  RowsIn q;
  RowsOut out;
  float* lse;  // nullable
  const int32_t* query_start;
  const int32_t* kv_len;
  float scale;
  int window;  // 0: none
  CacheView cache;
  int sinks;   // first tokens seen beside the window
  int groups;  // of requests that share their first tokens
  const int32_t* group_start;
  const int32_t* shared_len;
};

// How a call is divided: row_tile rows a workgroup, `tiles` workgroups for a
// request's rows, contexts in splits
// of split_len tokens (the last one takes what is left).  The parts of split s
// and row t, head h are at (s * T + t) * q_heads + h.
struct AttnPlan {
  int row_tile, tiles, split_len, num_splits;
  int first_part;   // of the call's splits, where several kernels' parts are joined
  size_t ml_bytes, o_bytes;
  float2* part_ml;  // maximum (base-2 logarithm), sum of weights
  float* part_o;    // weighted values
};
// even: contexts are short, and (nearly) of one length.
AttnPlan plan_attention(int B, int T, int q_heads, int kv_heads, int D, int max_q_len, int max_kv_len,
                        bool even = false);
hipError_t launch_attention(const AttnArgs& a, const AttnPlan& p, int cache_dtype, hipStream_t stream);

// With a window and first tokens that stay visible.
AttnPlan plan_sinks(int B, int T, int q_heads, int kv_heads, int D, int max_q_len, int max_kv_len, int window, int sinks);
hipError_t launch_sinks(const AttnArgs& a, const AttnPlan& p, int cache_dtype, hipStream_t stream);

// Behind tokens that groups of requests share: how those are divided, and each
// request's own, whose parts follow.
struct SharedPlan {
  AttnPlan shared, own;
  size_t bytes;
};
SharedPlan plan_shared(int B, int T, int groups, int q_heads, int kv_heads, int D, int max_q_len, int max_group_len,
                       int max_shared_len, int max_own_len);
hipError_t launch_shared(const AttnArgs& a, const SharedPlan& p, int cache_dtype, hipStream_t stream);

}  // namespace sv
