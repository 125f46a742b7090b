// Attention of requests whose first tokens are the same, which are read once for
// all of them.
//
// A group's requests follow each other, so their new rows do: the rows of a
// group are taken as one request's over the shared tokens (kShared), each
// request's rows over its own tokens (kOwn), both by the kernels of
// sv_attn_kernels.hpp, and a last kernel joins the parts of the two: with a
// part's maximum m, sum l and weighted values o of a row,
//   M = max m,  out = sum 2^(m - M) o / sum 2^(m - M) l.
//
// The rows of a group are many, which makes the shared part a matter of the
// matrix units, while a request's own tokens are read for a few rows only and
// are a matter of HBM: one launch (attn_shared_both.hip) has both at once.
//
// Measured, 32 query heads over 8 of 128 channels: 128 decoding requests behind
// 8000 shared tokens, own contexts of 125 to 500, 200 MB and 17 GFLOP in 65 + 8
// us (one after the other, and joined by a workgroup a row, 37 + 42 + 17);
// verification of 256 requests of 5 new tokens behind 8 prompts, 8-bit cache, 839
// MB and 90 GFLOP, 243 + 21 us (97 + 187 + 96); 8 samples behind 16000 tokens, 68
// MB in 24 + 6 us (22 + 8 + 6).  What is missing to the read rate: a compute unit
// has places for two workgroups of either kind, so that while the shared part
// runs the own one has half of its loads in flight.
//
// Where it does not pay: a row has two parts at least, written and read in
// binary32, and every request a workgroup of its own a head for its own tokens.
// Prompts (2048 new behind 4096: 296 us, sv_paged_attention 228), short shared
// parts (177 requests of 4 new behind 40 + 43: 42 and 16) and 256 channels (78
// behind 182 + 53: 55 and 38) are quicker without sharing.
//
// Registers: the few-rows kernels of 128 8-bit channels take 170 to 187 (16 rows),
// two waves a SIMD for the whole contexts' three; those of 256 bf16 channels spill
// up to 67 (few rows) and 41 (many rows, pages of fewer than 16 tokens).
#include "sv_attn_kernels.hpp"
#include "sv_attn_shared.hpp"

namespace sv {

namespace {

// The parts of a request's rows, as the kernels that wrote them saw them: those
// of the group's splits, and of its own live ones.
template <int M, int ALIGN>
struct PartsOf {
  const AttnArgs& a;
  const SharedPlan& p;
  int token0, next, len, before, shared;
  __device__ __forceinline__ PartsOf(const AttnArgs& a, const SharedPlan& p, int b, int token0, int next)
      : a(a), p(p), token0(token0), next(next) {
    len = max(uniform_at(a.kv_len, b), 0);
    before = shared_tokens_of(a, b);
    shared = before > 0 ? min((before - 1) / p.shared.split_len, p.shared.num_splits - 1) + 1 : 0;
  }
  // The i-th of a row's `parts` parts is the call's i-th (i < shared) or (first + i)-th.
  __device__ __forceinline__ void of(int tok, int head, int& parts, int& first) const {
    const int G = a.q_heads / a.cache.heads;
    const int64_t row = int64_t(tok - token0) * G + head % G;
    const Tile t =
        tile_of<M, Part::kOwn, ALIGN>(a, G, token0, int64_t(next) - token0, len, row / M * M, before);
    Splits live = {0, -1};
    if (t.rows != 0 && t.begin < t.end) live = live_splits(t, p.own.split_len, p.own.num_splits);
    parts = uniform(shared + live.last - live.first + 1);
    first = uniform(p.own.first_part + live.first - shared);
  }
};

// Joins the parts of a row's group and of its request: a wave takes `heads_at`
// heads of a token in turn, a lane 2 (above 128 channels 4) channels of all
// parts, whose weights the lanes form, one each, 64 parts at a time.
template <int M, int ALIGN, int CH>
__global__ __launch_bounds__(kAttnThreads) void join_shared_kernel(AttnArgs a, SharedPlan p, int heads_at) {
  typedef float Some __attribute__((ext_vector_type(CH)));
  const int lane = threadIdx.x & 63;
  const int D = a.cache.D;
  const int64_t all = int64_t(a.T) * a.q_heads;
  const int turns = (a.q_heads + heads_at - 1) / heads_at;  // of waves for a token
  const int64_t at_wave = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * kAttnWaves + uniform(threadIdx.x >> 6);
  const int tok = uniform(int(at_wave / turns)), head0 = uniform(int(at_wave % turns)) * heads_at;
  if (tok >= a.T) return;
  int token0, next;
  const int b = request_of(a, tok, uniform_at, token0, next);
  if (b < 0) return;
  const PartsOf<M, ALIGN> rows(a, p, b, token0, next);
  // (the same for all rows of a tile, of which a request mostly has one)
  const bool one_tile = int64_t(next - token0) * (a.q_heads / a.cache.heads) <= M;
  int parts, first;
  rows.of(tok, head0, parts, first);
  const int ch = min(CH * lane, D - CH);
  for (int head = head0; head < min(head0 + heads_at, a.q_heads); ++head) {
    const int64_t at = int64_t(tok) * a.q_heads + head;
    if (!one_tile) rows.of(tok, head, parts, first);
    const auto index = [&](int i) { return int64_t(i < rows.shared ? i : first + i) * all + at; };
    float top = -INFINITY, total = 0.f;
    Some y = 0.f;
    for (int from = 0; from < parts; from += 64) {
      const int n = min(parts - from, 64);
      // parts are asked for eight at a time, the first ones along with the statistics
      constexpr int kAhead = 8;
      Some v[kAhead];
      const auto ask = [&](int s) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (s + i < n) v[i] = *reinterpret_cast<const Some*>(p.own.part_o + index(from + s + i) * D + ch);
      };
      ask(0);
      const float2 ml = lane < n ? p.own.part_ml[index(from + lane)] : make_float2(-INFINITY, 0.f);
      float higher = ml.x;
#pragma unroll
      for (int i = 32; i >= 1; i >>= 1) higher = fmaxf(higher, __shfl_xor(higher, i, 64));
      higher = fmaxf(higher, top);
      const float ref = higher == -INFINITY ? 0.f : higher, keep = fast_exp2(top - ref);
      top = higher;
      const float weight = fast_exp2(ml.x - ref);
      total = fmaf(total, keep, wave_sum(weight * ml.y));
      y *= keep;
      for (int s = 0; s < n; s += kAhead) {
        if (s > 0) ask(s);
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (s + i < n) y += v[i] * __int_as_float(__builtin_amdgcn_readlane(__float_as_int(weight), s + i));
      }
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    if (CH * lane < D) {
      uint16_t* out = static_cast<uint16_t*>(a.out.p) + int64_t(tok) * a.out.token + head * a.out.head + ch;
#pragma unroll
      for (int i = 0; i < CH; i += 2) reinterpret_cast<uint32_t*>(out)[i / 2] = pack_bf16(y[i] * inv, y[i + 1] * inv);
    }
    if (a.lse && lane == 0) a.lse[at] = total == 0.f ? -INFINITY : (top + fast_log2(total)) * kLn2;
  }
}

// The same for few rows of many parts: a workgroup a row.
template <int M, int ALIGN>
__global__ __launch_bounds__(kAttnThreads) void join_few_shared_kernel(AttnArgs a, SharedPlan p) {
  __shared__ float4 sums[kAttnThreads];
  const int tok = blockIdx.x, head = blockIdx.y;
  int token0, next;
  const int b = request_of(a, tok, uniform_at, token0, next);
  if (b < 0) return;
  const PartsOf<M, ALIGN> row(a, p, b, token0, next);
  int parts, first;
  row.of(tok, head, parts, first);
  const int64_t at = int64_t(tok) * a.q_heads + head;
  if (parts > 0) {
    join_row(a, p.own, sums, at, parts, [&](int i) { return i < row.shared ? i : first + i; });
    return;
  }
  // a row that sees nothing
  const int ch = 4 * threadIdx.x;
  if (ch < a.cache.D)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out.p) + int64_t(tok) * a.out.token + head * a.out.head + ch) =
        make_uint2(0u, 0u);
  if (a.lse && threadIdx.x == 0) a.lse[at] = -INFINITY;
}

template <int M, int ALIGN>
void launch_join_shared(const AttnArgs& a, const SharedPlan& p, hipStream_t stream) {
  const int64_t rows = int64_t(a.T) * a.q_heads;
  // (8 requests of 32 heads with 64 parts: 6 us, a wave a row 11)
  if (rows <= 1024 && p.shared.num_splits + p.own.num_splits > 16) {
    hipLaunchKernelGGL((join_few_shared_kernel<M, ALIGN>), dim3(a.T, a.q_heads), dim3(kAttnThreads), 0, stream, a, p);
    return;
  }
  // several heads a wave, which then looks its request up once for them, where
  // the waves fill the card all the same (40960 rows of 2 parts: one 40 us, four
  // 22.6, eight 21.5; 17460 rows of 2 to 4 one 18, four 12; 4096 rows of 9 one 8)
  const int heads_at = rows <= 8192 ? 1 : rows <= 32768 ? 4 : 8;
  const int64_t waves = int64_t(a.T) * ((a.q_heads + heads_at - 1) / heads_at);
  // (threads of one dimension of a grid are counted in 32 bits)
  const int64_t blocks = (waves + kAttnWaves - 1) / kAttnWaves, wide = blocks < (1 << 22) ? blocks : 1 << 22;
  const dim3 grid(unsigned(wide), unsigned((blocks + wide - 1) / wide)), block(kAttnThreads);
  if (a.cache.D <= 128)
    hipLaunchKernelGGL((join_shared_kernel<M, ALIGN, 2>), grid, block, 0, stream, a, p, heads_at);
  else
    hipLaunchKernelGGL((join_shared_kernel<M, ALIGN, 4>), grid, block, 0, stream, a, p, heads_at);
}

}  // namespace

SharedPlan plan_shared(int B, int T, int groups, int q_heads, int kv_heads, int D, int max_q_len, int max_group_len,
                       int max_shared_len, int max_own_len) {
  SharedPlan p;
  p.shared = plan_attention(groups, T, q_heads, kv_heads, D, max_group_len, max_shared_len);
  if (p.shared.row_tile > 32) {
    // A workgroup a compute unit, as far as 256 tokens for each go: where the own
    // parts are in the same launch, theirs take the other places, and every split
    // is a part to be written and read (128 requests behind 8000: two a compute
    // unit 74 + 10 us, one 66 + 8, one for two 76 + 7).  Whole calls in us, so
    // and with the two a compute unit of plan_attention: 256 requests of 5 new
    // behind 8 prompts 252 and 278; one part after the other, 64 of 20 new behind
    // 8000 189 and 214, 88 of 10 behind 13236 248 and 307, 256 channels, 128 behind
    // 8000 171 and 191.  Against it: 19 of 22 new behind 11392 77 and 69, 4 of 512
    // behind 4096 216 and 208, 256 channels, 128 of 5 new 8-bit 449 and 389.
    const int64_t tiles = int64_t(groups) * p.shared.tiles * kv_heads;
    int64_t n = tiles > 0 ? (256 + tiles - 1) / tiles : 1;
    const int64_t most = (int64_t(max_shared_len) + 255) / 256;
    n = n < most ? n : most;
    if (n < p.shared.num_splits) {
      const int64_t len = n > 1 ? ((max_shared_len + n - 1) / n + 127) / 128 * 128 : max_shared_len;
      p.shared.split_len = int(len < 128 ? 128 : len);
      p.shared.num_splits = n > 1 ? int((int64_t(max_shared_len) + p.shared.split_len - 1) / p.shared.split_len) : 1;
    }
  }
  p.own = plan_attention(B, T, q_heads, kv_heads, D, max_q_len, max_own_len);
  p.own.first_part = p.shared.num_splits;
  const size_t rows = size_t(T) * q_heads, parts = size_t(p.shared.num_splits) + p.own.num_splits;
  const size_t ml = (parts * rows * sizeof(float2) + 255) / 256 * 256;
  p.own.ml_bytes = p.shared.ml_bytes = ml;
  p.bytes = ml + parts * rows * D * sizeof(float);
  return p;
}

hipError_t launch_shared(const AttnArgs& a, const SharedPlan& p, int cache_dtype, hipStream_t stream) {
  if (!launch_shared_and_own(a, p, cache_dtype, stream)) {
    launch_part<Part::kShared>(a, p.shared, cache_dtype, stream);
    launch_part<Part::kOwn>(a, p.own, cache_dtype, stream);
  }
  if (p.own.row_tile == 16)
    launch_join_shared<16, kBlock>(a, p, stream);
  else if (p.own.row_tile == 32)
    launch_join_shared<32, kBlock>(a, p, stream);
  else
    launch_join_shared<kManyRows, kTile>(a, p, stream);
  return hipGetLastError();
}

}  // namespace sv
