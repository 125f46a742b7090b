// Causal attention of packed new tokens over a paged cache: how a call is
// divided, and its launch (the kernels: sv_attn_kernels.hpp).
#include "sv_attn_kernels.hpp"

namespace sv {

// Bytes of divided contexts' parts.  (The rules that fill the card have at most
// 1024 tiles of 128 rows, 2048 of 32 or 4096 of 16: a quarter of it at most.)
constexpr size_t kMostParts = size_t(1) << 29;

AttnPlan plan_attention(int B, int T, int q_heads, int kv_heads, int D, int max_q_len, int max_kv_len, bool even) {
  AttnPlan p;
  const int G = q_heads / kv_heads;
  const int least = B > 0 ? (T + B - 1) / B : T;  // some request has that many rows
  max_q_len = max_q_len < least ? least : max_q_len > T ? T : max_q_len;
  if (max_kv_len > SV_ATTN_MAX_TOKENS) max_kv_len = SV_ATTN_MAX_TOKENS;  // no page table holds more (and sums stay in 32 bits)
  const int64_t rows = int64_t(max_q_len) * G;
  p.row_tile = rows <= 16 ? 16 : rows <= 32 ? 32 : kManyRows;
  // a request's tiles, as far as known; workgroups go on to further ones where
  // a request has more
  int64_t tiles = (rows + p.row_tile - 1) / p.row_tile;
  const int64_t most_tiles = (1 << 20) / (B > 0 ? B : 1);  // (tiles of all requests and heads: 32 bits)
  tiles = tiles < most_tiles ? tiles : most_tiles;
  p.tiles = int(tiles < 1 ? 1 : tiles);
  // Enough workgroups to fill the compute units twice over, of at least 256
  // tokens each; four times with two tiles of rows and eight times with one,
  // whose parts cost little, so that requests of different lengths even out (one:
  // 1024 to 4096 tokens in a batch of 64, 150 us filled twice, 138 us eight times;
  // two: 5 new tokens of 4 heads behind 100 to 8000, 16 requests 78 us filled
  // twice, 68 four times, 63 eight times, but equal lengths of 4096 61, 60 and 67).
  const int64_t groups = int64_t(B) * p.tiles * kv_heads;
  const int64_t want = p.row_tile == 16 ? 2048 : p.row_tile == 32 ? 1024 : 512;
  int64_t n = groups > 0 ? (want + groups - 1) / groups : 1;
  n = n < (max_kv_len + 255) / 256 ? n : (max_kv_len + 255) / 256;
  // With few of them one compute unit's reads are what counts (about 37 bytes a
  // nanosecond): a workgroup for every one then, down to 128 tokens each (8
  // heads of 1024 tokens: 8 workgroups 18.6 us, 32 of them 12.3, 64 of them
  // 10.5).  Up to 512 tokens joining costs as much as it saves.
  int64_t fine = groups > 0 ? 256 / groups : 1;
  fine = fine < (max_kv_len + 127) / 128 ? fine : (max_kv_len + 127) / 128;
  n = n > fine ? n : fine;
  // Ranges of at most 16384 tokens, in up to 8 splits: a long context among
  // many short ones does not wait for one workgroup then (one of 131000 tokens
  // among 255 of 1000: 2.0 -> 0.65 ms; 256 of 1000 where 131000 are allowed for,
  // 187 -> 225 us, where 32000 are, 194 us).  As many as their parts stay within
  // kMostParts: with more rows the short contexts take as long as the long one
  // (4096 requests of 5 tokens behind 700, 131000 allowed for: 2.7 GB of parts
  // and 2.89 ms with 8 splits, 2.26 with none; one of 131000 among them 3.51
  // and 3.88).
  const size_t rows_all = size_t(T) * q_heads;
  const size_t part_bytes = rows_all * (D * sizeof(float) + sizeof(float2));
  int64_t ranges = (max_kv_len + 16383) / 16384 < 8 ? (max_kv_len + 16383) / 16384 : 8;
  if (part_bytes * ranges > kMostParts) ranges = kMostParts / part_bytes;
  if (p.row_tile <= 32 && n < ranges) n = ranges;
  // Short contexts of one length need no more than the compute units' places, two
  // each, nearly filled once (64 requests of 8 heads that see 2052 tokens: 117 us
  // in 4 splits, 109 in one; of 5 8-bit new tokens 92 in two, 66 in one; 24 of 4100
  // tokens, which fill three eighths: 86 in 11, 92 in 3).
  if (even && groups >= 448) n = 1;
  if (n < 1 || max_kv_len <= 512) n = 1;
  int64_t len = (max_kv_len + n - 1) / n;
  len = (len + 127) / 128 * 128;
  p.split_len = int(len < 128 ? 128 : len);
  p.num_splits = int((int64_t(max_kv_len) + p.split_len - 1) / p.split_len);
  if (p.num_splits < 1) p.num_splits = 1;
  p.ml_bytes = p.num_splits > 1 ? (size_t(p.num_splits) * rows_all * sizeof(float2) + 255) / 256 * 256 : 0;
  p.o_bytes = p.num_splits > 1 ? (size_t(p.num_splits) * rows_all * D * sizeof(float) + 255) / 256 * 256 : 0;
  p.part_ml = nullptr;
  p.part_o = nullptr;
  p.first_part = 0;
  return p;
}

hipError_t launch_attention(const AttnArgs& a, const AttnPlan& p, int cache_dtype, hipStream_t stream) {
  launch_part<Part::kAll>(a, p, cache_dtype, stream);
  return hipGetLastError();
}

}  // namespace sv
