// Attention over a paged cache with a sliding window and a few first tokens that
// stay visible: the kernels of sv_attn_kernels.hpp over a range of tokens with a
// gap between the two.  Both ends of the gap lie on whole pieces of 32 (few rows)
// or 64 tokens, so that no load spans it; what a piece holds beyond the first
// tokens or before the window is masked.
//
// Bound as the kernels are: 64 requests of 7500 to 30000 bf16 tokens, window
// 2048 and 4 first tokens, 8 heads of 128 channels under 32 queries each, 539 MB
// in 107 us (4.95 TB/s); 2048 new tokens behind 8192 8-bit ones,
// window 4096 and 128 first tokens, 142 GFLOP in 158 to 168 us (840 to 900
// TFLOP/s); one token behind 100000, window 4096, 9 + 4 us (latency).
#include "sv_attn_kernels.hpp"

namespace sv {

// A tile of rows reads the first tokens, its window's and its own rows' at most:
// contexts are divided as if they were all as long as that (with the pieces of
// tokens that the ends of the two lie in), and no longer.
AttnPlan plan_sinks(int B, int T, int q_heads, int kv_heads, int D, int max_q_len, int max_kv_len, int window, int sinks) {
  const AttnPlan p = plan_attention(B, T, q_heads, kv_heads, D, max_q_len, max_kv_len);
  if (window == 0) return p;
  const int64_t reach = int64_t(window) + sinks + p.row_tile / (q_heads / kv_heads) + 2 * kTile;
  return reach < max_kv_len ? plan_attention(B, T, q_heads, kv_heads, D, max_q_len, int(reach), true) : p;
}

hipError_t launch_sinks(const AttnArgs& a, const AttnPlan& p, int cache_dtype, hipStream_t stream) {
  if (a.window == 0) return launch_attention(a, p, cache_dtype, stream);  // every row sees all before it
  launch_part<Part::kSinks>(a, p, cache_dtype, stream);
  return hipGetLastError();
}

}  // namespace sv
