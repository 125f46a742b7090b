// Attention over a paged cache with a sliding window and a few first tokens that
// stay visible: the kernels of sv_attn_kernels.hpp over a range of tokens with a
// gap between the two.  Both ends of the gap lie on whole pieces of 32 (few rows)
// or 64 tokens, so that no load spans it; what a piece holds beyond the first
// tokens or before the window is masked.
//
// Bound as the kernels are: 64 requests of 7500 to 30000 bf16 tokens, window
// 2048 and 4 first tokens, 8 heads of 128 channels under 32 queries in all, 539 MB
// in 107 us (4.95 TB/s); 128 such requests of 8-bit tokens, 544 MB, in 110 us a
// call, although the kernel of 16 rows and 128 8-bit channels takes 169 registers
// or 170, one or two more than let a third wave run on a SIMD; 2048 new tokens behind 8192 8-bit ones,
// window 4096 and 128 first tokens, 142 GFLOP in 158 to 168 us (840 to 900
// TFLOP/s); one token behind 100000, window 4096, 9 + 4 us (latency).
#include "sv_attn_kernels.hpp"

namespace sv {

// Tokens up to which a tile's reach makes contexts even, for each of its rows: a
// batch of 64 requests, 8 heads each, whose contexts are all longer than the
// window / of all lengths up to that / one as long and 63 of 300 tokens, in us,
// undivided and divided,
//   16 rows a tile (one new token, bf16)   32 rows (5 new tokens, 8-bit)
//   1024   54 39 28    58 46 34               35  27 22    64  49 34
//   2048  110 74 42   116 71 39               59  42 32    84  63 39
//   4096  207 154 69  206 133 52             119  87 50   141  99 49
//   8192  400 299 123 381 245 76             225 174 86   244 173 75
//  16384  787 593 234 735 470 120            438 336 160  439 310 118
// (and 65536 tokens, one row: 3116 2342 954, divided 2837 1762 350).
constexpr int kEvenTokensARow = 256;

// A tile of rows reads the first tokens, its window's and its own rows' at most:
// contexts are divided as if they were all as long as that (with the pieces of
// tokens that the ends of the two lie in), and no longer.
AttnPlan plan_sinks(int B, int T, int q_heads, int kv_heads, int D, int max_q_len, int max_kv_len, int window, int sinks) {
  const AttnPlan p = plan_attention(B, T, q_heads, kv_heads, D, max_q_len, max_kv_len);
  if (window == 0) return p;
  const int64_t reach = int64_t(window) + sinks + p.row_tile / (q_heads / kv_heads) + 2 * kTile;
  if (reach >= max_kv_len) return p;
  const bool even = reach <= int64_t(kEvenTokensARow) * (p.row_tile < 32 ? p.row_tile : 32);
  return plan_attention(B, T, q_heads, kv_heads, D, max_q_len, int(reach), even);
}

hipError_t launch_sinks(const AttnArgs& a, const AttnPlan& p, int cache_dtype, hipStream_t stream) {
  if (a.window == 0) return launch_attention(a, p, cache_dtype, stream);  // every row sees all before it
  launch_part<Part::kSinks>(a, p, cache_dtype, stream);
  return hipGetLastError();
}

}  // namespace sv
