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
};
hipError_t launch_append(const AppendArgs& a, int dtype, int cache_dtype, hipStream_t stream);

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
};

// How a call is divided: row_tile rows a workgroup, `tiles` workgroups for a
// request's rows, contexts in splits
// of split_len tokens (the last one takes what is left).  The parts of split s
// and row t, head h are at (s * T + t) * q_heads + h.
struct AttnPlan {
  int row_tile, tiles, split_len, num_splits;
  size_t ml_bytes, o_bytes;
  float2* part_ml;  // maximum (base-2 logarithm), sum of weights
  float* part_o;    // weighted values
};
AttnPlan plan_attention(int B, int T, int q_heads, int kv_heads, int D, int max_q_len, int max_kv_len);
hipError_t launch_attention(const AttnArgs& a, const AttnPlan& p, int cache_dtype, hipStream_t stream);

}  // namespace sv
