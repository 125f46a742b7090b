// Causal attention of packed new tokens over a paged cache.
//
// For a request b and key / value head kvh, the n new tokens and the
// G = q_heads / heads query heads of the group make R = n * G rows that read
// the same keys and values: row r is token r / G, head kvh * G + r % G.  A
// workgroup takes a tile of rows and a range of tokens (a split) and forms, for
// a row with scores x_j = scale q . k_j,
//   l = sum_j exp(x_j - m),   o = sum_j exp(x_j - m) v_j,   out = o / l,
// in one pass over the tokens with a running reference m near the maximum.
//
// Scores are formed transposed, S^T = K Q^T, so that a lane of the matrix
// instruction's result holds one row and several tokens: the softmax
// statistics of a row are one value per lane, its running maximum a reduction
// inside the lane and over the lanes of the row, and the weights are already
// the B operand of O^T += V^T P^T (the order of the tokens inside a product's
// inner dimension is free as long as both operands agree).  Only V^T needs its
// elements transposed, which the transposing LDS reads do.
//
// Few rows (up to 32 a request and head: decoding, verification of drafts):
// HBM-bound. The four waves take blocks of 32 tokens in turn, each with its
// own running statistics, so that no wave waits for another until their
// results are joined at the end; keys go from memory to registers directly in
// the A operand's layout (a lane's 16 bytes of one token's row), values
// through the wave's own part of LDS. A wave asks for the next block's keys
// and values as soon as the present ones have left their registers. Measured:
// 64 requests of 1024 to 4096 bf16 tokens, 8 heads of 128 channels, 677 MB
// read in 135 us (5.0 TB/s, of which the paged rows alone read at 6.1 in a
// kernel that only loads); 256 requests of 500 to 2000 8-bit tokens, 5 new
// tokens of 4 heads for each of 8, 689 MB in 149 us (4.6 TB/s). What is
// missing to the read rate: a workgroup's start and end (5 to 7 us each, in
// which its compute unit slot asks for nothing) and the uneven lengths at the
// end of the grid.
//
// Many rows (chunks of a prompt): bound by the softmax's vector instructions
// and by LDS, both beside the products. The four waves have 32 rows each and
// share tiles of 64 tokens, loaded a tile ahead into registers and staged in
// two LDS buffers, so that a tile is read from memory once for 128 rows.
// Measured: 2048 new tokens behind 8192, 32 heads of 128 channels over 8: 309
// GFLOP in 331 to 336 us, 920 to 934 TFLOP/s (library products of two 4096 x
// 4096 and two 8192 x 8192 matrices: 1087 and 1278); packed prompts of up to
// 4000 tokens at 64 channels with a window of 2048, where a product has half
// the work for each exponential: 612 TFLOP/s. With a tile of rows a request it
// is HBM-bound as well: 9 new tokens of 8 heads for each of 4 behind 131071, 4
// requests, 1.07 GB in 213 us (5.0 TB/s). 20 rows of 256 channels (5 tokens of
// 4 heads) are about as fast in either kernel for bf16 (72.8 and 74.9 us, 16
// requests of 2048 tokens), but not for 8-bit caches (46.8 and 67.0 us).
//
// Splits: where rows are few and contexts long, a context is divided into
// ranges of `split_len` tokens, whose results (running maximum, sum, weighted
// values in binary32) a second kernel joins.
#pragma once

#include "sv_attn.hpp"

namespace sv {

namespace {

constexpr int kAttnThreads = 256;
constexpr int kAttnWaves = kAttnThreads / 64;
constexpr int kBlock = 32;  // tokens a wave takes at a time
// Weights are taken relative to a running maximum that follows the true one only
// when that is more than 2^8 ahead: sums and weights then stay far inside binary32
// and bf16, and the accumulated values are rescaled in a few blocks instead of
// in nearly all (some row of a tile has a new maximum in almost every one):
// 2048 new tokens behind 8192 344 -> 334 us, packed prompts 211 -> 202 us.
constexpr float kSlack = 8.f;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// Values that every lane of a workgroup reads alike (lengths, page tables) go
// through the scalar cache: a vector load would wait behind the streamed keys
// and values of the compute unit.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int32_t uniform_at(const int32_t* p, int64_t i) {
  return ((const __attribute__((address_space(4))) int32_t*)(p))[i];
}

// 16 bytes at a scalar address plus a lane's 32-bit offset.  The offset is made
// opaque here so that the load takes both as they are, instead of a 64-bit
// vector address formed ahead and kept in registers.
__device__ __forceinline__ uint4 load_from(const char* p, uint32_t at) {
  asm volatile("" : "+v"(at));
  return *reinterpret_cast<const uint4*>(p + at);
}

// Workgroups go to the 8 XCDs in turn, and an XCD's to its 4 shader engines in
// turn, so that one of these 32 would get the same requests for every head and
// split, and requests of different lengths load them unevenly.  The requests
// are therefore turned by 9 places (an XCD and an engine) from head to head, by
// 27 from split to split: 64 contexts of 1024 to 4096 tokens, shuffled or
// ascending, 156 and 146 -> 138 us; 4 of 2000 to 60000, 148 -> 84 us.
struct Block {
  uint32_t x, y, z, nx;  // a workgroup's place in its grid, and the grid's width
};
__device__ __forceinline__ uint32_t spread_over_xcds(const Block& at) {
  return (at.x + 9u * at.y + 27u * at.z) % at.nx;
}
__device__ __forceinline__ Block this_block() { return {blockIdx.x, blockIdx.y, blockIdx.z, gridDim.x}; }

// Which tokens of its request a row takes.  A tile of rows counts the tokens of
// its range from `begin` to `end`; in kSinks and kOwn, where the range has a gap,
// those from `skip_at` on stand for tokens `skip` further on (both multiples of
// the tokens taken at a time, so that no such piece spans the gap).
enum class Part {
  kAll,     // j <= place, and j > place - window with a window
  kSinks,   // the same, and j < sinks with a window: the gap lies between first tokens and window
  kShared,  // j <= place among the shared tokens of a group, whose requests' rows are taken as one request's
  kOwn      // j <= place among the tokens behind them: the gap is what is shared
};
constexpr bool is_whole(Part part) { return part == Part::kAll || part == Part::kSinks; }

// One tile of rows of one request (kShared: of one group).
struct Tile {
  int first_row;   // tile's first row in the request (row = token * G + head in group)
  int rows;        // rows of the tile; 0: nothing to do
  int token0;      // the request's first packed row
  int place0;      // place of the request's first new token
  int begin, end;  // tokens that some row of the tile may see
  int skip_at, skip;
  int before;      // kOwn: the shared tokens
  int request;     // whose row of the page table is read
};

__device__ __forceinline__ int token_at(Part part, const Tile& t, int base) {
  return part == Part::kSinks ? base + (base >= t.skip_at ? t.skip : 0) : part == Part::kOwn ? base + t.skip : base;
}

// The tokens that group g shares, as far as a page table can hold them.
template <typename Load>
__device__ __forceinline__ int shared_tokens(const AttnArgs& a, int g, Load load) {
  return int(min(int64_t(max(load(a.shared_len, g), 0)), int64_t(a.cache.max_pages) << a.cache.page_shift));
}

// Whether a group of the requests first .. next - 1 is within the batch: no other
// shares anything, neither where its tokens are read nor where its parts are joined.
__device__ __forceinline__ bool group_stands(const AttnArgs& a, int first, int next) {
  return first >= 0 && first < next && next <= a.B;
}

// The tokens that request b shares: those of the group that it is in, if any.
// Groups of equally many requests are found at once, others by a search of the
// whole wave.
__device__ __forceinline__ int shared_tokens_of(const AttnArgs& a, int b) {
  int g = int(int64_t(b) * a.groups / a.B);
  int first = uniform_at(a.group_start, g), next = uniform_at(a.group_start, g + 1);
  const int shared = shared_tokens(a, g, uniform_at);
  if (b >= first && b < next) return group_stands(a, first, next) ? shared : 0;
  g = uniform(find_sequence(a.group_start, a.groups, b, threadIdx.x & 63));
  if (g < 0) return 0;
  first = uniform_at(a.group_start, g), next = uniform_at(a.group_start, g + 1);
  return b < next && group_stands(a, first, next) ? shared_tokens(a, g, uniform_at) : 0;
}

// The tile of a request of n rows from token0 on and len cached tokens, the
// first `before` of them shared (kOwn), whose first row is first_row; rows == 0
// beyond the request's last.  ALIGN: tokens taken at a time.
template <int M, Part PART, int ALIGN>
__device__ __forceinline__ Tile tile_of(const AttnArgs& a, int G, int token0, int64_t n, int64_t len,
                                        int64_t first_row, int before) {
  Tile t;
  t.rows = 0;
  t.token0 = token0;
  t.skip_at = t.skip = 0;
  t.before = before;
  const int64_t rows = n * G - first_row;
  if (t.token0 < 0 || int64_t(t.token0) + n > a.T || rows <= 0) return t;
  t.first_row = int(first_row);
  t.rows = int(min(rows, int64_t(M)));
  const int64_t held = min(len, int64_t(a.cache.max_pages) << a.cache.page_shift);
  const int64_t place0 = len - n;
  t.place0 = int(place0);
  const int64_t first_place = place0 + t.first_row / G, last_place = place0 + (t.first_row + t.rows - 1) / G;
  t.end = int(max(int64_t(0), min(held, last_place + 1)));
  t.begin = a.window > 0 ? int(min(int64_t(t.end), max(int64_t(0), first_place - a.window + 1))) : 0;
  if constexpr (PART == Part::kSinks) {
    const int reach = t.begin & ~(ALIGN - 1);  // the window's first token, or one before
    t.skip_at = int(min((int64_t(a.sinks) + ALIGN - 1) & ~int64_t(ALIGN - 1), int64_t(reach)));
    t.skip = reach - t.skip_at;
    t.begin = 0;
    t.end -= t.skip;
  } else if constexpr (PART == Part::kOwn) {
    t.skip = min(before, t.end) & ~(ALIGN - 1);
    t.begin = min(before, t.end) - t.skip;
    t.end -= t.skip;
  }
  return t;
}

// The same of request b (kShared: of group b), for the whole workgroup.
template <int M, Part PART, int ALIGN>
__device__ __forceinline__ Tile tile_at(const AttnArgs& a, int G, int b, int64_t first_row) {
  Tile t;
  if constexpr (PART == Part::kShared) {
    const int first = uniform_at(a.group_start, b), next = uniform_at(a.group_start, b + 1);
    t.rows = 0;
    if (!group_stands(a, first, next)) return t;
    const int token0 = uniform_at(a.query_start, first);
    const int64_t n = int64_t(uniform_at(a.query_start, next)) - token0, rows = n * G - first_row;
    if (token0 < 0 || int64_t(token0) + n > a.T || rows <= 0) return t;
    t.first_row = int(first_row);
    t.rows = int(min(rows, int64_t(M)));
    t.token0 = token0;
    t.request = first;
    t.begin = 0;
    t.end = shared_tokens(a, b, uniform_at);
  } else {
    const int token0 = uniform_at(a.query_start, b), len = max(uniform_at(a.kv_len, b), 0);
    t = tile_of<M, PART, ALIGN>(a, G, token0, int64_t(uniform_at(a.query_start, b + 1)) - token0, len, first_row,
                                PART == Part::kOwn ? shared_tokens_of(a, b) : 0);
    t.request = b;
    t.place0 = uniform(t.place0);
    if constexpr (!(PART == Part::kAll)) t.skip_at = uniform(t.skip_at), t.skip = uniform(t.skip);
  }
  // 64-bit comparisons are vector instructions: back to scalars
  t.token0 = uniform(t.token0), t.rows = uniform(t.rows), t.first_row = uniform(t.first_row);
  t.begin = uniform(t.begin), t.end = uniform(t.end);
  return t;
}

// The place of a packed row of group g: requests of equally many rows are found
// at once, others by a search.
__device__ __forceinline__ int place_in_group(const AttnArgs& a, int g, int row) {
  const int first = uniform_at(a.group_start, g), next = uniform_at(a.group_start, g + 1);
  const int from = uniform_at(a.query_start, first), to = uniform_at(a.query_start, next);
  int b = first + int(int64_t(row - from) * (next - first) / (to - from));
  int end = a.query_start[b + 1];
  if (row < a.query_start[b] || row >= end) {
    int hi = next;  // the last request that starts at the row or before is b - 1 in the end
    for (b = first; b < hi;) {
      const int mid = b + ((hi - b) >> 1);
      if (a.query_start[mid] <= row)
        b = mid + 1;
      else
        hi = mid;
    }
    end = a.query_start[max(b, first + 1)];
    b = max(b - 1, first);
  }
  return max(a.kv_len[b], 0) - (end - row);
}

// Byte offset of a page's token in keys or values: strides in units of 16 bytes.
__device__ __forceinline__ uint64_t row_at(const UnitStrides& u, int page, int slot, int head) {
  return ((uint64_t(uint32_t(page)) * u.page + uint64_t(uint32_t(slot)) * u.token) + uint64_t(uint32_t(head)) * u.head)
         << 4;
}

// The splits that have tokens of [begin, end): first .. last (empty: 0 .. 0).
struct Splits {
  int first, last;
};
__device__ __forceinline__ Splits live_splits(const Tile& t, int split_len, int num_splits) {
  if (t.begin >= t.end) return {0, 0};
  return {min(t.begin / split_len, num_splits - 1), min((t.end - 1) / split_len, num_splits - 1)};
}

// Bits 15 and 31 tell whether a packed bf16 is infinite or NaN (an exponent of
// ones carries into its sign).
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) { return (w & 0x7f807f80u) + 0x00800080u; }
__device__ __forceinline__ uint32_t not_finite8(const uint4& w) {
  return (not_finite2(w.x) | not_finite2(w.y) | not_finite2(w.z) | not_finite2(w.w)) & 0x80008000u;
}

// A value, or zeros.
__device__ __forceinline__ uint4 only_if(bool keep, const uint4& w) {
  return make_uint4(keep ? w.x : 0u, keep ? w.y : 0u, keep ? w.z : 0u, keep ? w.w : 0u);
}

// The larger of a value and that of the lane 32 away, or 16 and 32 away.
__device__ __forceinline__ float max_over_halves(float x) {
  const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1]));
}
__device__ __forceinline__ float max_over_quarters(float x) {
  const auto y = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return max_over_halves(fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1])));
}

// Nothing moves across: left alone, the compiler reads a product's operand from
// LDS right before its use and waits for it.
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0); }

__device__ __forceinline__ f32x4 mfma16(const uint4& a, const uint4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}

// 4 x 16 elements of LDS transposed: each group of 16 lanes reads 4 rows of 16
// bf16 (lane i the 4 from column 4 (i % 4) of row i / 4) and gets column i.
__device__ __forceinline__ uint2 read_transposed(const uint16_t* p) {
  const s16x4 r = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) s16x4*)(const_cast<uint16_t*>(p)));
  return __builtin_bit_cast(uint2, r);
}

// Elements between rows in LDS.  The 16 bytes beyond a row of keys set
// successive rows off by one 16-byte unit, so that 8 rows' units of the same
// channels (a load of the A operand) lie on different banks; a transposing read
// takes 32 bytes of 4 rows at a time, which 32 bytes beyond a row keep apart.
// (The few-rows kernel stores its values 16 rows at a time, for which 16 bytes
// are as good on balance.)  The addresses stay sums, whose constant parts are
// the instructions' offsets.
template <int DP>
constexpr int kPitch = DP + 8;
template <int DP>
constexpr int kValuePitch = DP + 16;

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------

// SMALL: pages of fewer than 16 tokens (or rows too far apart for a 32-bit
// offset within 16 tokens): every lane looks its token's page up.  Otherwise 16
// tokens lie in one page, whose address is scalar.
template <int DP>
using FewValues = uint16_t[kAttnWaves][kBlock * kPitch<DP>];
template <int MT>
using FewStats = float[kAttnWaves][16 * MT];

template <int DP, int MT, bool FP8, bool SMALL, Part PART>
__device__ __forceinline__ void few_rows(const AttnArgs& a, const AttnPlan& p, FewValues<DP>& values,
                                         FewStats<MT>& stat_m, FewStats<MT>& stat_l, const Block& block) {
  constexpr int M = 16 * MT;
  constexpr int kSteps = DP / 32;        // of the score product
  constexpr int kDT = DP / 16;           // channel tiles of the result
  constexpr int kLoads = FP8 ? DP / 64 : DP / 32;  // 16-byte loads of a token's row per lane

  const CacheView& c = a.cache;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int kvh = block.y, split = block.z;
  const int G = a.q_heads / c.heads;
  const int at_x = spread_over_xcds(block);
  const int b = at_x / p.tiles;
  for (int64_t first_row = int64_t(at_x - b * p.tiles) * M;; first_row += int64_t(p.tiles) * M) {
    const Tile t = tile_at<M, PART, kBlock>(a, G, b, first_row);
    if (t.rows == 0) return;
    const Splits live = live_splits(t, p.split_len, p.num_splits);
    if (split < live.first || split > live.last || (!is_whole(PART) && t.begin >= t.end)) continue;
    const int begin = max(t.begin, split * p.split_len) & ~(kBlock - 1);
    const int end = split == p.num_splits - 1 ? t.end : min(t.end, (split + 1) * p.split_len);
    const int last = token_at(PART, t, end - 1);

    // queries: the B operand, lane (row, g) holding the channels of its steps
    const int chunks = c.D >> 3;
    uint4 qf[MT][kSteps];
    int place[MT], oldest[MT];  // of the lane's rows: they see the tokens oldest < j <= place
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row = 16 * m + r;
      const int tok = (t.first_row + row) / G, head = kvh * G + (t.first_row + row) % G;
      if constexpr (PART != Part::kShared) place[m] = row < t.rows ? t.place0 + tok : -1;
      oldest[m] = PART == Part::kOwn ? t.before - 1 : a.window > 0 ? max(place[m], -1) - a.window : -1;
      const uint16_t* q = static_cast<const uint16_t*>(a.q.p) + int64_t(t.token0 + tok) * a.q.token + head * a.q.head;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int ch = FP8 ? 8 * (s >> 1) + 2 * g + (s & 1) : 4 * s + g;
        qf[m][s] = make_uint4(0u, 0u, 0u, 0u);
        if (row < t.rows && ch < chunks) qf[m][s] = *reinterpret_cast<const uint4*>(q + 8 * ch);
      }
    }
    // the places of the tile's first and last rows (kShared: whether some row does not see all)
    int first_place = 0, last_place = 0;
    if constexpr (PART != Part::kShared) {
      first_place = t.place0 + t.first_row / G;
      last_place = t.place0 + (t.first_row + t.rows - 1) / G;
    }
    const float sc = a.scale * kLog2e;

    f32x4 o[kDT][MT];
    float mx[MT], l[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      mx[m] = -INFINITY;
      l[m] = 0.f;
#pragma unroll
      for (int d = 0; d < kDT; ++d) o[d][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    uint4 kr[2][kLoads], vr[2][kLoads];
    uint32_t ks[2] = {127, 127}, vs[2] = {127, 127};
    bool have[2];
    const int64_t table = t.request * c.table_stride;
    const int in_page = (1 << c.page_shift) - 1;
    // the page table's entries of the block's tokens 0 .. 15 and 16 .. 31 (SMALL:
    // of this lane's, r and 16 + r), or of the last token in their place
    int page[2];
    auto pages = [&](int base) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = min(token_at(PART, t, base) + 16 * h + (SMALL ? r : 0), last);
        page[h] = SMALL ? c.table[table + (j >> c.page_shift)] : uniform_at(c.table, table + (j >> c.page_shift));
      }
    };
    // ask for a block's rows; the loads of absent tokens and of channels beyond
    // the head's go to page 0 and to its last channels: the tokens are not seen,
    // the keys' channels made zero, the values' not stored
    uint32_t lane_at[2][kLoads];  // bytes from the 16 tokens' first row, of keys and of values
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint32_t unit = min(4 * i + g, (FP8 ? c.D >> 4 : c.D >> 3) - 1);
      lane_at[0][i] = (uint32_t(SMALL ? 0 : r) * c.ku.token + unit) << 4;
      lane_at[1][i] = (uint32_t(SMALL ? 0 : r) * c.vu.token + unit) << 4;
    }
    uint32_t lanes = ~0u;
    auto request = [&](int base, const void* p0, const UnitStrides& u, const uint32_t (&at_lane)[kLoads],
                       const uint8_t* scale, uint4 (&in)[2][kLoads], uint32_t (&in_scale)[2]) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = uint32_t(page[h]) < uint32_t(c.num_pages) ? page[h] : 0;
        const int slot = (token_at(PART, t, base) + 16 * h + (SMALL ? r : 0)) & in_page;
        const char* q = static_cast<const char*>(p0) + row_at(u, at, slot, kvh);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) in[h][i] = load_from(q, at_lane[i] & lanes);
        if (FP8) in_scale[h] = scale[((int64_t(at) * c.heads + kvh) << c.page_shift) + slot + (SMALL ? 0 : r)];
      }
    };
    auto request_keys = [&](int base) { request(base, c.k, c.ku, lane_at[0], c.k_scale, kr, ks); };
    auto request_values = [&](int base) {
      request(base, c.v, c.vu, lane_at[1], c.v_scale, vr, vs);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        have[h] = uint32_t(page[h]) < uint32_t(c.num_pages) && base + 16 * h + r < end;
    };

    const int stride = kAttnWaves * kBlock;
    int base = begin + wave * kBlock;
    uint16_t* const mine = values[wave];
    if (base < end) {
      pages(base);
      request_keys(base);
      request_values(base);
      pages(base + stride < end ? base + stride : base);
      if constexpr (PART == Part::kShared) {  // (looked up while the first keys and values are on their way)
        bool low = false;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int row = 16 * m + r;
          place[m] = row < t.rows ? place_in_group(a, b, t.token0 + (t.first_row + row) / G) : -1;
          low |= row < t.rows && place[m] < t.end - 1;
        }
        first_place = __any(low) ? -1 : INT32_MAX;
      }
      do {
        // the queries are zero beyond the head's channels, but zero times an infinite key would be NaN
        if (c.D < DP) {
          int beyond = lane >> 4;
          asm volatile("" : "+v"(beyond));  // (masks formed here, not kept in registers through the loop)
          beyond -= FP8 ? c.D >> 4 : c.D >> 3;
#pragma unroll
          for (int i = 0; i < kLoads; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) kr[h][i] = only_if(beyond + 4 * i < 0, kr[h][i]);
        }
        // S^T, a block's 16 tokens by 16 rows at a time
        f32x4 s[2][MT];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int m = 0; m < MT; ++m) s[h][m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int st = 0; st < kSteps; ++st)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint4 kf;
            if (FP8) {
              const uint4 w = kr[h][st >> 1];
              kf = dequant8((st & 1) ? make_uint2(w.z, w.w) : make_uint2(w.x, w.y), scale_of(ks[h]));
            } else {
              kf = kr[h][st];
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) s[h][m] = mfma16(kf, qf[m][st], s[h][m]);
          }
        // Behind the wave's last block every lane asks for one word of the same
        // block again, which nothing reads: loads on one path only would have to be
        // waited for as if on the other.
        const bool more = base + stride < end;
        const int next = more ? base + stride : base;
        lanes = more ? ~0u : 0u;
        request_keys(next);
        // every row sees every token of the block, unless it reaches beyond the
        // first row's place or the last row's window, or lacks tokens
        const int token = token_at(PART, t, base);
        bool in_reach = a.window == 0 || token > last_place - a.window;
        if constexpr (PART == Part::kSinks) in_reach |= token + kBlock <= a.sinks;
        if constexpr (PART == Part::kShared) in_reach = true;
        if constexpr (PART == Part::kOwn) in_reach = token >= t.before;
        const bool whole = __all(have[0] && have[1]) && token + kBlock - 1 <= first_place && in_reach;
        uint32_t hidden = 0, nan = 0;  // bit 16 h + i: token 16 h + i is absent; its value is not finite
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint16_t* const to = mine + (16 * h + r) * kPitch<DP> + (FP8 ? 16 : 8) * g;
          uint32_t bad = 0;
#pragma unroll
          for (int i = 0; i < kLoads; ++i) {
            if (FP8) {
              const float vscale = scale_of(vs[h]);
              const uint4 lo = dequant8(make_uint2(vr[h][i].x, vr[h][i].y), vscale);
              const uint4 hi = dequant8(make_uint2(vr[h][i].z, vr[h][i].w), vscale);
              *reinterpret_cast<uint4*>(to + 64 * i) = lo;
              *reinterpret_cast<uint4*>(to + 64 * i + 8) = hi;
              if (!whole) bad |= not_finite8(lo) | not_finite8(hi);
            } else {
              *reinterpret_cast<uint4*>(to + 32 * i) = vr[h][i];
              if (!whole) bad |= not_finite8(vr[h][i]);
            }
          }
          if (!whole) {
            // a weight of zero does not stop a value that is not finite: such
            // values are taken out, and their tokens' scores made NaN instead
            uint64_t any = __ballot(bad != 0 && have[h]);
            any |= any >> 32;
            any |= any >> 16;
            nan |= uint32_t(any & 0xffffu) << (16 * h);
            hidden |= uint32_t(~__ballot(have[h]) & 0xffffu) << (16 * h);
            asm volatile("" ::: "memory");  // (a store of its own: else every value would be chosen in registers first)
            if (!have[h] || ((any >> r) & 1u)) {
#pragma unroll
              for (int i = 0; i < kLoads; ++i) {
                *reinterpret_cast<uint4*>(to + (FP8 ? 64 : 32) * i) = make_uint4(0u, 0u, 0u, 0u);
                if (FP8) *reinterpret_cast<uint4*>(to + 64 * i + 8) = make_uint4(0u, 0u, 0u, 0u);
              }
            }
          }
        }
        request_values(next);
        pages(next + stride < end ? next + stride : next);
        if (!whole) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int k = 16 * h + 4 * g + i, j = token + k;
              const bool off = (hidden >> k) & 1u, bad = (nan >> k) & 1u;
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                const bool sees = !off & (j <= place[m]) & ((j > oldest[m]) | (PART == Part::kSinks && j < a.sinks));
                const float x = bad ? NAN : s[h][m][i];
                s[h][m][i] = sees ? x : -INFINITY;
              }
            }
        }
        // values are read from LDS four channel tiles ahead of their products
        uint4 vf[2][4];
        const uint16_t* const vt = mine + (4 * g + (r >> 2)) * kPitch<DP> + 4 * (r & 3);
        auto read_values = [&](int d) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint2 v0 = read_transposed(vt + 16 * (d + i));
            const uint2 v1 = read_transposed(vt + 16 * kPitch<DP> + 16 * (d + i));
            vf[(d >> 2) & 1][i] = make_uint4(v0.x, v0.y, v1.x, v1.y);
          }
        };
        read_values(0);
        // weights, in place of the scores, and the running statistics
        uint4 pf[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          float top = -INFINITY;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, s[h][m][i]);
          top = max_over_quarters(top);
          const bool ahead = (top - mx[m]) * sc > kSlack;
          if (__any(ahead)) {
            const float higher = ahead ? top : mx[m];  // (one row's scores change no other row's roundings)
            const float keep = fast_exp2((mx[m] - (higher == -INFINITY ? 0.f : higher)) * sc);
            mx[m] = higher;
            l[m] *= keep;
#pragma unroll
            for (int d = 0; d < kDT; ++d) o[d][m] *= keep;
          }
          const float ref = mx[m] == -INFINITY ? 0.f : mx[m] * sc;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              s[h][m][i] = fast_exp2(fmaf(s[h][m][i], sc, -ref));
              l[m] += s[h][m][i];
            }
          // rounded to bf16 for the product: a weight is off by at most 2^-8 of itself
          pf[m] = make_uint4(pack_bf16(s[0][m][0], s[0][m][1]), pack_bf16(s[0][m][2], s[0][m][3]),
                             pack_bf16(s[1][m][0], s[1][m][1]), pack_bf16(s[1][m][2], s[1][m][3]));
        }
#pragma unroll
        for (int d = 0; d < kDT; d += 4) {
          if (d + 4 < kDT) read_values(d + 4);
          keep_order();
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < MT; ++m) o[d + i][m] = mfma16(vf[(d >> 2) & 1][i], pf[m], o[d + i][m]);
          keep_order();
        }
        base += stride;
      } while (base < end);
    }

    // join the waves: the tile's maximum, then each wave's results scaled to it
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      l[m] += __shfl_xor(l[m], 16, 64);
      l[m] += __shfl_xor(l[m], 32, 64);
      if (g == 0) {
        stat_m[wave][16 * m + r] = mx[m];
        stat_l[wave][16 * m + r] = l[m];
      }
    }
    __syncthreads();
    const bool alone = is_whole(PART) && live.first == live.last;
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));  // (what follows from it is formed here, not kept in registers through the loop)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (16 * m >= t.rows) break;
      const int row = 16 * m + r;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kAttnWaves; ++w) top = fmaxf(top, stat_m[w][row]);
      const float ref = top == -INFINITY ? 0.f : top * sc;
      const float keep = fast_exp2(fmaf(mx[m], sc, -ref));
      // rows of DP channels and 16 bytes more, which keep 8 rows' stores apart
      float* part = reinterpret_cast<float*>(values[wave]) + r * (DP + 4) + 4 * g;
#pragma unroll
      for (int d = 0; d < kDT; ++d)
        *reinterpret_cast<float4*>(part + 16 * d) =
            make_float4(o[d][m][0] * keep, o[d][m][1] * keep, o[d][m][2] * keep, o[d][m][3] * keep);
      __syncthreads();
      // 16 rows by 16 threads, 8 channels at a time
      const int orow = tid >> 4;
      const int trow = 16 * m + orow;
      if (trow < t.rows) {
        float rtop = -INFINITY, total = 0.f;
#pragma unroll
        for (int w = 0; w < kAttnWaves; ++w) rtop = fmaxf(rtop, stat_m[w][trow]);
        const float rref = rtop == -INFINITY ? 0.f : rtop * sc;
#pragma unroll
        for (int w = 0; w < kAttnWaves; ++w) total += stat_l[w][trow] * fast_exp2(fmaf(stat_m[w][trow], sc, -rref));
        const int tok = t.token0 + (t.first_row + trow) / G, head = kvh * G + (t.first_row + trow) % G;
        const int64_t at = int64_t(tok) * a.q_heads + head;
        const float inv = total == 0.f ? 0.f : 1.f / total;
        for (int ch = tid & 15; ch < chunks; ch += 16) {
          float y[8] = {};
#pragma unroll
          for (int w = 0; w < kAttnWaves; ++w) {
            float x[8];
            load8(reinterpret_cast<const float*>(values[w]) + orow * (DP + 4) + 8 * ch, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] += x[j];
          }
          if (alone) {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] *= inv;
          }
          if (alone)
            store8(static_cast<uint16_t*>(a.out.p) + int64_t(tok) * a.out.token + head * a.out.head + 8 * ch, y);
          else
            store8(p.part_o + ((p.first_part + split) * (int64_t(a.T) * a.q_heads) + at) * c.D + 8 * ch, y);
        }
        if ((tid & 15) == 0) {
          if (!alone)
            p.part_ml[(p.first_part + split) * (int64_t(a.T) * a.q_heads) + at] =
                make_float2(rtop == -INFINITY ? rtop : rref, total);
          else if (a.lse)
            a.lse[at] = total == 0.f ? -INFINITY : (rref + fast_log2(total)) * kLn2;
        }
      }
      __syncthreads();
    }
  }
}

template <int DP, int MT, bool FP8, bool SMALL, Part PART>
__global__ __launch_bounds__(kAttnThreads, DP == 256 ? 1 : DP * MT >= 128 ? 2 : 3) void few_rows_kernel(
    AttnArgs a, AttnPlan p) {
  __shared__ __align__(16) FewValues<DP> values;
  __shared__ FewStats<MT> stat_m, stat_l;
  few_rows<DP, MT, FP8, SMALL, PART>(a, p, values, stat_m, stat_l, this_block());
}

// ---------------------------------------------------------------------------
// many rows
// ---------------------------------------------------------------------------

typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16 mfma32(const uint4& a, const uint4& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}

constexpr int kTile = 64;      // tokens of a tile
constexpr int kManyRows = 32 * kAttnWaves;

// PAGES: 0 pages of fewer than 16 tokens (or rows too far apart for a 32-bit
// offset), every thread looks its tokens' pages up; 1 a load's tokens of a wave
// lie in one page; 2 the tile lies in one page.
template <int DP>
using ManyKeys = uint16_t[2][kTile * kPitch<DP>];
template <int DP>
using ManyValues = uint16_t[2][kTile * kValuePitch<DP>];
using ManyState = uint8_t[2][kTile];    // of a token: 0 present, 1 absent, 2 a value not finite
using ManyMarks = int[2][kAttnWaves];   // some token that this wave loaded has a state

template <int DP, bool FP8, int PAGES, Part PART>
__device__ __forceinline__ void many_rows(const AttnArgs& a, const AttnPlan& p, ManyKeys<DP>& keys,
                                          ManyValues<DP>& values, ManyState& state, ManyMarks& marks,
                                          const Block& block) {
  constexpr int M = kManyRows;
  constexpr int kSteps = DP / 16;
  constexpr int kDT = DP / 32;
  constexpr int kLanes = FP8 ? DP / 16 : DP / 8;  // that load a token's row, 16 bytes each
  constexpr int kSpan = kAttnThreads / kLanes;    // tokens of one load of the workgroup
  constexpr int kWaveSpan = 64 / kLanes;          // and of a wave
  constexpr int kLoads = kTile / kSpan;
  constexpr int kParts = FP8 ? 2 : 1;             // 8 channels each, of a load
  constexpr int kGroup = DP == 64 ? 2 : 4;        // products whose operands are read together

  const CacheView& c = a.cache;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int r = lane & 31, h = lane >> 5;
  const int split = block.z;
  const int G = a.q_heads / c.heads;
  // workgroups go to the 8 XCDs in turn: each takes whole heads, whose keys and
  // values then pass through one L2 only
  uint32_t at_x = block.x, kvh = block.y;
  if ((c.heads & 7) == 0) {
    const uint32_t i = block.x + block.y * block.nx, per = block.nx * (c.heads >> 3);
    const uint32_t pos = (i & 7) * per + (i >> 3);
    kvh = pos / block.nx;
    at_x = pos - kvh * block.nx;
  } else {
    at_x = spread_over_xcds(block);
  }
  const int b = at_x / p.tiles;
  // later tiles of a prompt see more: they start first
  for (int64_t first_row = int64_t(p.tiles - 1 - (at_x - b * p.tiles)) * M;; first_row += int64_t(p.tiles) * M) {
    const Tile t = tile_at<M, PART, kTile>(a, G, b, first_row);
    if (t.rows == 0) return;
    const Splits live = live_splits(t, p.split_len, p.num_splits);
    if (split < live.first || split > live.last || (!is_whole(PART) && t.begin >= t.end)) continue;
    const int begin = max(t.begin, split * p.split_len) & ~(kTile - 1);
    const int end = split == p.num_splits - 1 ? t.end : min(t.end, (split + 1) * p.split_len);
    const int last = token_at(PART, t, end - 1);

    int place;
    uint4 qf[kSteps];
    {
      const int row = 32 * wave + r;
      const int tok = (t.first_row + row) / G, head = kvh * G + (t.first_row + row) % G;
      const uint16_t* q = static_cast<const uint16_t*>(a.q.p) + int64_t(t.token0 + tok) * a.q.token + head * a.q.head;
      if constexpr (PART == Part::kShared)
        place = row < t.rows ? place_in_group(a, b, t.token0 + tok) : -1;
      else
        place = row < t.rows ? t.place0 + tok : -1;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        qf[s] = make_uint4(0u, 0u, 0u, 0u);
        if (row < t.rows && 8 * (2 * s + h) < c.D) qf[s] = *reinterpret_cast<const uint4*>(q + 8 * (2 * s + h));
      }
    }
    const float sc = a.scale * kLog2e;
    const bool busy = 32 * wave < t.rows;
    int oldest;  // the row sees the tokens oldest < j <= place
    // the places of the wave's first and last rows, and the last tokens before their windows
    int first_place, last_oldest, wave_first, wave_last, wave_oldest, wave_newest;
    if constexpr (PART == Part::kShared) {  // (whether some row of the tile, of the wave, does not see all)
      const bool low = 32 * wave + r < t.rows && place < t.end - 1;
      oldest = last_oldest = wave_oldest = wave_newest = -1;
      first_place = __syncthreads_or(low) ? -1 : INT32_MAX;
      wave_first = __any(low) ? -1 : INT32_MAX;
      wave_last = INT32_MAX;
    } else {
      first_place = t.place0 + t.first_row / G;
      const int last_place = t.place0 + (t.first_row + t.rows - 1) / G;
      wave_first = uniform(t.place0 + (t.first_row + 32 * wave) / G);
      wave_last = uniform(t.place0 + (t.first_row + min(32 * wave + 31, t.rows - 1)) / G);
      if constexpr (PART == Part::kOwn) {
        oldest = last_oldest = wave_oldest = wave_newest = t.before - 1;
      } else {
        oldest = a.window > 0 ? max(place, -1) - a.window : -1;
        last_oldest = a.window > 0 ? max(last_place, -1) - a.window : -1;
        wave_oldest = a.window > 0 ? max(wave_first, -1) - a.window : -1;
        wave_newest = a.window > 0 ? max(wave_last, -1) - a.window : -1;
      }
    }

    f32x16 o[kDT];
#pragma unroll
    for (int d = 0; d < kDT; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
    float mx = -INFINITY, l = 0.f;

    // staging: thread -> token kSpan * i + tid / kLanes, 16 bytes tid % kLanes
    uint4 kin[kLoads], vin[kLoads];
    uint32_t kscale[kLoads], vscale[kLoads];
    int page[PAGES == 2 ? 1 : kLoads];  // page table entries: of the tile, of the wave's loads, of the thread's tokens
    const int64_t table = t.request * c.table_stride;
    const int in_page = (1 << c.page_shift) - 1;
    const int own = PAGES == 0 ? tid / kLanes : wave * kWaveSpan;  // of a load's tokens, the first that `page` is of
    const int from = PAGES == 0 ? 0 : lane / kLanes;               // this thread's token behind it
    const uint32_t unit = min(tid % kLanes, (FP8 ? c.D >> 4 : c.D >> 3) - 1);
    auto pages = [&](int base) {
      if constexpr (PAGES == 2) {
        page[0] = uniform_at(c.table, table + (min(token_at(PART, t, base), last) >> c.page_shift));
      } else {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int j = min(token_at(PART, t, base) + kSpan * i + own, last) >> c.page_shift;
          page[i] = PAGES == 0 ? c.table[table + j] : uniform_at(c.table, table + j);
        }
      }
    };
    auto found = [&](int i) { return uint32_t(page[PAGES == 2 ? 0 : i]) < uint32_t(c.num_pages); };
    auto request = [&](int base, const void* p0, const UnitStrides& u, const uint8_t* scale, uint4 (&in)[kLoads],
                       uint32_t (&in_scale)[kLoads]) {
      const uint32_t lane_at = (uint32_t(from) * u.token + unit) << 4;  // bytes from the row of `own`
      if constexpr (PAGES == 2) {
        const int at = found(0) ? page[0] : 0, slot = (token_at(PART, t, base) + own) & in_page;
        const char* q = static_cast<const char*>(p0) + row_at(u, at, slot, kvh);
        const uint8_t* so = FP8 ? scale + ((int64_t(at) * c.heads + kvh) << c.page_shift) + slot : scale;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          in[i] = load_from(q, lane_at);
          q += uint64_t(u.token) * kSpan << 4;
          if (FP8) in_scale[i] = so[kSpan * i + from];
        }
      } else {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int at = found(i) ? page[i] : 0, slot = (token_at(PART, t, base) + kSpan * i + own) & in_page;
          in[i] = load_from(static_cast<const char*>(p0) + row_at(u, at, slot, kvh), lane_at);
          if (FP8) in_scale[i] = scale[((int64_t(at) * c.heads + kvh) << c.page_shift) + slot + from];
        }
      }
    };
    // every row of the tile sees all 64 tokens, as far as places go
    auto whole = [&](int base) {
      const int token = token_at(PART, t, base);
      bool in_reach = token > last_oldest;
      if constexpr (PART == Part::kSinks) in_reach |= token + kTile <= a.sinks;
      return token + kTile - 1 <= first_place && base + kTile <= end && in_reach;
    };
    auto stage_keys = [&](int buf) {
      uint16_t* const to = &keys[buf][tid / kLanes * kPitch<DP> + 8 * kParts * (tid % kLanes)];
      // the queries are zero beyond the head's channels, but zero times an infinite key would be NaN
      if (c.D < DP) {
        int at = tid % kLanes;
        asm volatile("" : "+v"(at));  // (the mask formed here, not kept in registers through the loop)
#pragma unroll
        for (int i = 0; i < kLoads; ++i) kin[i] = only_if(at < (FP8 ? c.D >> 4 : c.D >> 3), kin[i]);
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        if (FP8) {
          const float scale = scale_of(kscale[i]);
          *reinterpret_cast<uint4*>(to + kSpan * i * kPitch<DP>) = dequant8(make_uint2(kin[i].x, kin[i].y), scale);
          *reinterpret_cast<uint4*>(to + kSpan * i * kPitch<DP> + 8) = dequant8(make_uint2(kin[i].z, kin[i].w), scale);
        } else {
          *reinterpret_cast<uint4*>(to + kSpan * i * kPitch<DP>) = kin[i];
        }
      }
    };
    int marked = 0;  // bit buf: this wave has left marks in state[buf] and marks[buf]
    auto stage_values = [&](int base, int buf) {
      const bool ok = whole(base);
      uint16_t* const to = &values[buf][tid / kLanes * kValuePitch<DP> + 8 * kParts * (tid % kLanes)];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        if (FP8) {
          const float scale = scale_of(vscale[i]);
          *reinterpret_cast<uint4*>(to + kSpan * i * kValuePitch<DP>) = dequant8(make_uint2(vin[i].x, vin[i].y), scale);
          *reinterpret_cast<uint4*>(to + kSpan * i * kValuePitch<DP> + 8) =
              dequant8(make_uint2(vin[i].z, vin[i].w), scale);
        } else {
          *reinterpret_cast<uint4*>(to + kSpan * i * kValuePitch<DP>) = vin[i];
        }
      }
      bool lack = false;
#pragma unroll
      for (int i = 0; i < (PAGES == 2 ? 1 : kLoads); ++i) lack |= !found(i);
      const bool trouble = !ok || (PAGES == 0 ? __any(lack) : lack);
      if (!trouble && !((marked >> buf) & 1)) return;
      // (from here on what was stored is read back: values kept for this in
      // registers would cost the usual path)
      asm volatile("" ::: "memory");
      bool some = false;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int at = kSpan * i + tid / kLanes;
        const bool gone = !found(i) || base + at >= end;
        // a weight of zero does not stop a value that is not finite: such
        // values are taken out, and their tokens' scores made NaN instead
        uint32_t bad = 0;
#pragma unroll
        for (int q = 0; q < kParts; ++q)
          bad |= not_finite8(*reinterpret_cast<const uint4*>(to + kSpan * i * kValuePitch<DP> + 8 * q));
        const uint64_t any = __ballot(bad != 0 && !gone);
        const bool spoiled = (any >> (lane & ~(kLanes - 1))) & ((uint64_t(1) << kLanes) - 1);
        if (gone || spoiled) {
#pragma unroll
          for (int q = 0; q < kParts; ++q)
            *reinterpret_cast<uint4*>(to + kSpan * i * kValuePitch<DP> + 8 * q) = make_uint4(0u, 0u, 0u, 0u);
        }
        if (tid % kLanes == 0) state[buf][at] = gone ? 1 : spoiled ? 2 : 0;
        some |= gone || spoiled;
      }
      some = __any(some);
      if (lane == 0) marks[buf][wave] = some;
      marked = trouble ? marked | (1 << buf) : marked & ~(1 << buf);
    };

    // (the barrier that ended the loop has ended every read of a former tile)
    if (tid < kTile) state[0][tid] = state[1][tid] = 0;
    if (tid < kAttnWaves) marks[0][tid] = marks[1][tid] = 0;
    __syncthreads();
    int buf = 0;
    if (begin < end) {
      pages(begin);
      request(begin, c.k, c.ku, c.k_scale, kin, kscale);
      request(begin, c.v, c.vu, c.v_scale, vin, vscale);
      stage_keys(0);
      stage_values(begin, 0);
      pages(begin + kTile);
    }
    __syncthreads();
    // One tile: its successor is asked for first and staged last (behind the
    // last tile the same slots of the last page, which nothing reads), without
    // a branch on the way that would hold the loads up.
    for (int base = begin; base < end; base += kTile) {
      const int next = base + kTile;
      request(next, c.k, c.ku, c.k_scale, kin, kscale);
      request(next, c.v, c.vu, c.v_scale, vin, vscale);
      // a wave without rows, or whose rows do not reach this far, only helps to load
      const int token = token_at(PART, t, base);
      if (busy && token <= wave_last && (token + kTile - 1 > wave_oldest || (PART == Part::kSinks && token < a.sinks))) {
        f32x16 s[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[u][i] = 0.f;
        // products in groups whose operands are read a group ahead; a wave
        // that has products to issue goes before one in its softmax (343 -> 334 us)
        {
          const uint16_t* const kt = &keys[buf][r * kPitch<DP> + 8 * h];
          uint4 kf[2][kGroup];
          auto read = [&](int n) {
#pragma unroll
            for (int i = 0; i < kGroup; ++i)
              kf[n / kGroup & 1][i] =
                  *reinterpret_cast<const uint4*>(kt + 32 * ((n + i) & 1) * kPitch<DP> + 16 * ((n + i) >> 1));
          };
          read(0);
          __builtin_amdgcn_s_setprio(1);
#pragma unroll
          for (int n = 0; n < 2 * kSteps; n += kGroup) {
            if (n + kGroup < 2 * kSteps) read(n + kGroup);
            keep_order();
#pragma unroll
            for (int i = 0; i < kGroup; ++i)
              s[(n + i) & 1] = mfma32(kf[n / kGroup & 1][i], qf[(n + i) >> 1], s[(n + i) & 1]);
            keep_order();
          }
        }
        __builtin_amdgcn_s_setprio(0);
        // scores of absent tokens, of values taken out, and of tokens that the row does not see
        const int4 mark = *reinterpret_cast<const int4*>(marks[buf]);
        if ((mark.x | mark.y | mark.z | mark.w) != 0) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t w = *reinterpret_cast<const uint32_t*>(&state[buf][32 * u + 8 * k + 4 * h]);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t is = (w >> (8 * i)) & 0xffu;
                if (is != 0) s[u][4 * k + i] = is == 1 ? -INFINITY : NAN;
              }
            }
        }
        if (token + kTile - 1 > wave_first) {
          const int upto = place - token - 4 * h;
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (32 * u + 8 * (i >> 2) + (i & 3) > upto) s[u][i] = -INFINITY;
        }
        if (token <= wave_newest && !(PART == Part::kSinks && token + kTile <= a.sinks)) {
          const int past = oldest - token - 4 * h;
          const int first = PART == Part::kSinks ? a.sinks - token - 4 * h : INT32_MIN;  // the first token's place that is no sink's
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (32 * u + 8 * (i >> 2) + (i & 3) <= past && 32 * u + 8 * (i >> 2) + (i & 3) >= first) s[u][i] = -INFINITY;
        }
        float top = -INFINITY;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) top = fmaxf(top, s[u][i]);
        top = max_over_halves(top);
        const bool ahead = (top - mx) * sc > kSlack;
        if (__any(ahead)) {
          const float higher = ahead ? top : mx;  // (one row's scores change no other row's roundings)
          const float keep = fast_exp2((mx - (higher == -INFINITY ? 0.f : higher)) * sc);
          mx = higher;
          l *= keep;
#pragma unroll
          for (int d = 0; d < kDT; ++d) o[d] *= keep;
        }
        const float ref = mx == -INFINITY ? 0.f : mx * sc;
        const uint16_t* const vt =
            &values[buf][(4 * h + ((lane & 15) >> 2)) * kValuePitch<DP> + (lane & 16) + 4 * (lane & 3)];
        uint4 vf[2][kGroup];
        auto read_values = [&](int n) {
#pragma unroll
          for (int i = 0; i < kGroup; ++i) {
            const int at = n + i, d = at % kDT, t16 = at / kDT;  // channels 32 d .., tokens 16 t16 ..
            const uint2 v0 = read_transposed(vt + 16 * t16 * kValuePitch<DP> + 32 * d);
            const uint2 v1 = read_transposed(vt + (16 * t16 + 8) * kValuePitch<DP> + 32 * d);
            vf[n / kGroup & 1][i] = make_uint4(v0.x, v0.y, v1.x, v1.y);
          }
        };
        read_values(0);
        uint4 pf[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            s[u][i] = fast_exp2(fmaf(s[u][i], sc, -ref));
            l += s[u][i];
          }
          // rounded to bf16 for the product: a weight is off by at most 2^-8 of itself
#pragma unroll
          for (int q = 0; q < 2; ++q)
            pf[u][q] = make_uint4(pack_bf16(s[u][8 * q], s[u][8 * q + 1]), pack_bf16(s[u][8 * q + 2], s[u][8 * q + 3]),
                                  pack_bf16(s[u][8 * q + 4], s[u][8 * q + 5]),
                                  pack_bf16(s[u][8 * q + 6], s[u][8 * q + 7]));
        }
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int n = 0; n < 4 * kDT; n += kGroup) {
          if (n + kGroup < 4 * kDT) read_values(n + kGroup);
          keep_order();
#pragma unroll
          for (int i = 0; i < kGroup; ++i) {
            const int at = n + i, d = at % kDT, t16 = at / kDT;
            o[d] = mfma32(vf[n / kGroup & 1][i], pf[t16 >> 1][t16 & 1], o[d]);
          }
          keep_order();
        }
        __builtin_amdgcn_s_setprio(0);
      }
      stage_keys(buf ^ 1);
      stage_values(next, buf ^ 1);
      pages(next + kTile);
      buf ^= 1;
      __syncthreads();
    }

    l += __shfl_xor(l, 32, 64);
    int row = 32 * wave + r;
    asm volatile("" : "+v"(row));  // (what follows from it is formed here, not kept in registers through the loop)
    if (row >= t.rows) continue;
    const int tok = t.token0 + (t.first_row + row) / G, head = kvh * G + (t.first_row + row) % G;
    const float ref = mx == -INFINITY ? 0.f : mx * sc;
    const int64_t at = int64_t(tok) * a.q_heads + head;
    if (is_whole(PART) && live.first == live.last) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      uint16_t* out = static_cast<uint16_t*>(a.out.p) + int64_t(tok) * a.out.token + head * a.out.head;
#pragma unroll
      for (int d = 0; d < kDT; ++d)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int e = 32 * d + 8 * k + 4 * h;
          if (e < c.D)
            *reinterpret_cast<uint2*>(out + e) = make_uint2(pack_bf16(o[d][4 * k] * inv, o[d][4 * k + 1] * inv),
                                                            pack_bf16(o[d][4 * k + 2] * inv, o[d][4 * k + 3] * inv));
        }
      if (a.lse && h == 0) a.lse[at] = l == 0.f ? -INFINITY : (ref + fast_log2(l)) * kLn2;
    } else {
      const int64_t part = (p.first_part + split) * (int64_t(a.T) * a.q_heads) + at;
#pragma unroll
      for (int d = 0; d < kDT; ++d)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int e = 32 * d + 8 * k + 4 * h;
          if (e < c.D)
            *reinterpret_cast<float4*>(p.part_o + part * c.D + e) =
                make_float4(o[d][4 * k], o[d][4 * k + 1], o[d][4 * k + 2], o[d][4 * k + 3]);
        }
      if (h == 0) p.part_ml[part] = make_float2(mx == -INFINITY ? mx : ref, l);
    }
  }
}

template <int DP, bool FP8, int PAGES, Part PART>
__global__ __launch_bounds__(kAttnThreads, DP > 128 ? 1 : DP > 64 ? 2 : 3) void many_rows_kernel(
    AttnArgs a, AttnPlan p) {
  __shared__ __align__(16) ManyKeys<DP> keys;
  __shared__ __align__(16) ManyValues<DP> values;
  __shared__ __align__(16) ManyState state;
  __shared__ __align__(16) ManyMarks marks;
  many_rows<DP, FP8, PAGES, PART>(a, p, keys, values, state, marks, this_block());
}

// ---------------------------------------------------------------------------
// joining splits
// ---------------------------------------------------------------------------

// Joins `parts` parts, the i-th of which is the index(i)-th of the call's, for
// the row `at` (of a token and a head), by the whole workgroup: every wave
// forms the row's maximum and sum from the parts' (a lane each); then groups of
// 32 (64 above 128 channels) lanes take the parts in turn, four channels a
// lane, and are added in LDS.
template <typename Index>
__device__ __forceinline__ void join_row(const AttnArgs& a, const AttnPlan& p, float4* sums, int64_t at, int parts,
                                         Index index) {
  const CacheView& c = a.cache;
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t all = int64_t(a.T) * a.q_heads;
  // the first parts are asked for along with the statistics
  constexpr int kAhead = 4;
  const int lg = c.D <= 128 ? 5 : 6, groups = kAttnThreads >> lg;
  const int ch = min(4 * (tid & ((1 << lg) - 1)), c.D - 4), first = tid >> lg;
  auto part_at = [&](int i) { return *reinterpret_cast<const float4*>(p.part_o + (index(i) * all + at) * c.D + ch); };
  float4 v[kAhead];
  float m[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int s = min(first + i * groups, parts - 1);
    v[i] = part_at(s);
    m[i] = p.part_ml[index(s) * all + at].x;
  }
  float top = -INFINITY;
  for (int s = lane; s < parts; s += 64) top = fmaxf(top, p.part_ml[index(s) * all + at].x);
#pragma unroll
  for (int i = 32; i >= 1; i >>= 1) top = fmaxf(top, __shfl_xor(top, i, 64));
  const float ref = top == -INFINITY ? 0.f : top;
  float total = 0.f;
  for (int s = lane; s < parts; s += 64) {
    const float2 ml = p.part_ml[index(s) * all + at];
    total = fmaf(fast_exp2(ml.x - ref), ml.y, total);
  }
  total = wave_sum(total);
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float4& x, float w) {
    y.x = fmaf(w, x.x, y.x), y.y = fmaf(w, x.y, y.y), y.z = fmaf(w, x.z, y.z), y.w = fmaf(w, x.w, y.w);
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (first + i * groups < parts) add(v[i], fast_exp2(m[i] - ref));
#pragma unroll 4
  for (int s = first + kAhead * groups; s < parts; s += groups)
    add(part_at(s), fast_exp2(p.part_ml[index(s) * all + at].x - ref));
  sums[tid] = y;
  __syncthreads();
  if (tid >> lg == 0) {
    for (int i = 1; i < groups; ++i) {
      const float4 x = sums[tid + (i << lg)];
      y.x += x.x, y.y += x.y, y.z += x.z, y.w += x.w;
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    if (4 * tid < c.D)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out.p) + at / a.q_heads * a.out.token +
                                at % a.q_heads * a.out.head + ch) =
          make_uint2(pack_bf16(y.x * inv, y.y * inv), pack_bf16(y.z * inv, y.w * inv));
    if (a.lse && tid == 0) a.lse[at] = total == 0.f ? -INFINITY : (ref + fast_log2(total)) * kLn2;
  }
  __syncthreads();
}

// The request of a packed row `tok`, its first row and its end in token0 and
// next; -1: it is of no request.  Requests of equally many rows are found at
// once, others by a search.
template <typename Load>
__device__ __forceinline__ int request_of(const AttnArgs& a, int tok, Load load, int& token0, int& next) {
  int b = int(int64_t(tok) * a.B / a.T);
  token0 = load(a.query_start, b), next = load(a.query_start, b + 1);
  if (tok >= token0 && tok < next) return b;
  int hi = a.B;  // the last request that starts at tok or before is b - 1 in the end
  for (b = 0; b < hi;) {
    const int mid = b + ((hi - b) >> 1);
    if (load(a.query_start, mid) <= tok)
      b = mid + 1;
    else
      hi = mid;
  }
  if (--b < 0) return -1;
  token0 = load(a.query_start, b), next = load(a.query_start, b + 1);
  return tok < next ? b : -1;
}

// A workgroup takes `per` rows: each lane looks up whether one of them was
// split, and those that were are joined in turn (a single row is looked up
// through the scalar cache, 2 us sooner).
// Bound by latency (a launch, the lengths, the parts, an LDS exchange): 10 us for
// 2048 rows of 4 splits and for 1152 of 32, 5 us for a single token's.
template <int M, Part PART, int ALIGN>
__global__ __launch_bounds__(kAttnThreads) void join_kernel(AttnArgs a, AttnPlan p, int per) {
  __shared__ float4 sums[kAttnThreads];
  const int lane = threadIdx.x & 63;
  const int G = a.q_heads / a.cache.heads;
  const int64_t all = int64_t(a.T) * a.q_heads, from = int64_t(blockIdx.x) * per, to = min(from + per, all);
  // the splits of a row of ours, as the kernel that wrote the parts saw them
  auto splits_of = [&](int64_t at, auto load) {
    const int tok = int(at / a.q_heads), head = int(at % a.q_heads);
    int token0, next;
    const int b = request_of(a, tok, load, token0, next);
    if (b < 0) return Splits{0, 0};
    const int64_t row = int64_t(tok - token0) * G + head % G;
    const Tile t =
        tile_of<M, PART, ALIGN>(a, G, token0, int64_t(next) - token0, max(load(a.kv_len, b), 0), row / M * M, 0);
    return t.rows != 0 ? live_splits(t, p.split_len, p.num_splits) : Splits{0, 0};
  };
  for (int64_t some = from; some < to; some += 64) {
    Splits mine = {0, 0};
    if (per == 1)
      mine = splits_of(blockIdx.x, uniform_at);
    else if (some + lane < to)
      mine = splits_of(some + lane, [](const int32_t* x, int64_t i) { return x[i]; });
    // (a row with one split was written by the split itself)
    for (uint64_t left = __ballot(mine.first != mine.last && some + lane < to); left != 0; left &= left - 1) {
      const int k = __builtin_ctzll(left);
      const Splits live = {__builtin_amdgcn_readlane(mine.first, k), __builtin_amdgcn_readlane(mine.last, k)};
      join_row(a, p, sums, some + k, live.last - live.first + 1, [&](int i) { return live.first + i; });
    }
  }
}

// Up to 4096 workgroups, twice what the card holds: where few of many rows were
// split, a workgroup for each would cost more than the joining (164 thousand
// rows: 250 us).  (Shared and own parts are joined together, attn_shared.hip.)
template <int M, Part PART, int ALIGN>
void launch_join(const AttnArgs& a, const AttnPlan& p, hipStream_t stream) {
  if constexpr (is_whole(PART)) {
    if (p.num_splits == 1) return;
    const int64_t all = int64_t(a.T) * a.q_heads;
    const int per = int((all + 4095) / 4096);
    const dim3 grid(int((all + per - 1) / per)), block(kAttnThreads);
    hipLaunchKernelGGL((join_kernel<M, PART, ALIGN>), grid, block, 0, stream, a, p, per);
  }
}

template <int DP, int MT, bool FP8, bool SMALL, Part PART>
void launch_few(const AttnArgs& a, const AttnPlan& p, const dim3& grid, hipStream_t stream) {
  hipLaunchKernelGGL((few_rows_kernel<DP, MT, FP8, SMALL, PART>), grid, dim3(kAttnThreads), 0, stream, a, p);
  launch_join<16 * MT, PART, kBlock>(a, p, stream);
}

template <int DP, bool FP8, bool SMALL, Part PART>
void launch_rows(const AttnArgs& a, const AttnPlan& p, hipStream_t stream) {
  const dim3 grid((PART == Part::kShared ? a.groups : a.B) * p.tiles, a.cache.heads, p.num_splits);
  if (p.row_tile == 16) {
    launch_few<DP, 1, FP8, SMALL, PART>(a, p, grid, stream);
  } else if (p.row_tile == 32) {
    launch_few<DP, 2, FP8, SMALL, PART>(a, p, grid, stream);
  } else {
    if (SMALL)
      hipLaunchKernelGGL((many_rows_kernel<DP, FP8, 0, PART>), grid, dim3(kAttnThreads), 0, stream, a, p);
    else if (a.cache.page_shift < 6)
      hipLaunchKernelGGL((many_rows_kernel<DP, FP8, 1, PART>), grid, dim3(kAttnThreads), 0, stream, a, p);
    else
      hipLaunchKernelGGL((many_rows_kernel<DP, FP8, 2, PART>), grid, dim3(kAttnThreads), 0, stream, a, p);
    launch_join<kManyRows, PART, kTile>(a, p, stream);
  }
}

template <bool FP8, bool SMALL, Part PART>
void launch_dims(const AttnArgs& a, const AttnPlan& p, hipStream_t stream) {
  if (a.cache.D <= 64)
    launch_rows<64, FP8, SMALL, PART>(a, p, stream);
  else if (a.cache.D <= 128)
    launch_rows<128, FP8, SMALL, PART>(a, p, stream);
  else
    launch_rows<256, FP8, SMALL, PART>(a, p, stream);
}

// Whether 16 tokens may lie in several pages, or farther apart than 2^32 bytes.
bool looks_up_each_token(const CacheView& c) {
  const auto near = [](const UnitStrides& u) { return u.token < (uint32_t(1) << 24); };
  return c.page_shift < 4 || !near(c.ku) || !near(c.vu);
}

template <Part PART>
void launch_part(const AttnArgs& a, const AttnPlan& p, int cache_dtype, hipStream_t stream) {
  const bool small = looks_up_each_token(a.cache);
  if (cache_dtype == SV_E4M3)
    small ? launch_dims<true, true, PART>(a, p, stream) : launch_dims<true, false, PART>(a, p, stream);
  else
    small ? launch_dims<false, true, PART>(a, p, stream) : launch_dims<false, false, PART>(a, p, stream);
}

}  // namespace

}  // namespace sv
