// Attention of requests whose first tokens are the same, which are read once for
// all of them.
//
// A group's requests follow each other, so their new rows do: the rows of a
// group are taken as one request's over the shared tokens (kShared), each
// request's rows over its own tokens (kOwn), both by the kernels of
// sv_attn_kernels.hpp, and a third kernel joins the parts of the two: with a
// part's maximum m, sum l and weighted values o of row r,
//   M = max m,  out = sum 2^(m - M) o / sum 2^(m - M) l.
#include "sv_attn_kernels.hpp"

namespace sv {

namespace {

// Joins the parts of a row's group and of its request.
template <int M, int ALIGN>
__global__ __launch_bounds__(kAttnThreads) void join_shared_kernel(AttnArgs a, SharedPlan p, int per) {
  __shared__ float4 sums[kAttnThreads];
  const int lane = threadIdx.x & 63;
  const int G = a.q_heads / a.cache.heads;
  const int64_t all = int64_t(a.T) * a.q_heads, from = int64_t(blockIdx.x) * per, to = min(from + per, all);
  // a row's parts: of the group's splits, and of its request's own from the first live one on
  struct Parts {
    int shared, own, first;
  };
  auto parts_of = [&](int64_t at, auto load) {
    const int tok = int(at / a.q_heads), head = int(at % a.q_heads);
    int token0, next;
    const int b = request_of(a, tok, load, token0, next);
    if (b < 0) return Parts{-1, 0, 0};
    Parts out = {0, 0, 0};
    int before = 0, hi = a.groups, g = 0;  // the last group that starts at b or before is g - 1 in the end
    while (g < hi) {
      const int mid = g + ((hi - g) >> 1);
      if (load(a.group_start, mid) <= b)
        g = mid + 1;
      else
        hi = mid;
    }
    if (--g >= 0 && b < load(a.group_start, g + 1)) {
      before = shared_tokens(a, g, load);
      if (before > 0) out.shared = min((before - 1) / p.shared.split_len, p.shared.num_splits - 1) + 1;
    }
    const int64_t row = int64_t(tok - token0) * G + head % G;
    const Tile t = tile_of<M, Part::kOwn, ALIGN>(a, G, token0, int64_t(next) - token0, max(load(a.kv_len, b), 0),
                                                 row / M * M, before);
    if (t.rows != 0 && t.begin < t.end) {
      const Splits live = live_splits(t, p.own.split_len, p.own.num_splits);
      out.own = live.last - live.first + 1;
      out.first = p.own.first_part + live.first;
    }
    return out;
  };
  for (int64_t some = from; some < to; some += 64) {
    Parts mine = {-1, 0, 0};
    if (per == 1)
      mine = parts_of(blockIdx.x, uniform_at);
    else if (some + lane < to)
      mine = parts_of(some + lane, [](const int32_t* x, int64_t i) { return x[i]; });
    for (uint64_t left = __ballot(mine.shared >= 0 && some + lane < to); left != 0; left &= left - 1) {
      const int k = __builtin_ctzll(left);
      const int shared = __builtin_amdgcn_readlane(mine.shared, k), own = __builtin_amdgcn_readlane(mine.own, k);
      const int first = __builtin_amdgcn_readlane(mine.first, k) - shared;
      const int64_t at = some + k;
      if (shared + own > 0) {
        join_row(a, p.own, sums, at, shared + own, [&](int i) { return i < shared ? i : first + i; });
        continue;
      }
      // a row that sees nothing
      const int ch = 4 * threadIdx.x;
      if (ch < a.cache.D)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out.p) + at / a.q_heads * a.out.token +
                                  at % a.q_heads * a.out.head + ch) = make_uint2(0u, 0u);
      if (a.lse && threadIdx.x == 0) a.lse[at] = -INFINITY;
    }
  }
}

template <int M, int ALIGN>
void launch_join_shared(const AttnArgs& a, const SharedPlan& p, hipStream_t stream) {
  const int64_t all = int64_t(a.T) * a.q_heads;
  const int per = int((all + 4095) / 4096);
  hipLaunchKernelGGL((join_shared_kernel<M, ALIGN>), dim3(int((all + per - 1) / per)), dim3(kAttnThreads), 0, stream, a,
                     p, per);
}

}  // namespace

SharedPlan plan_shared(int B, int T, int groups, int q_heads, int kv_heads, int D, int max_q_len, int max_group_len,
                       int max_shared_len, int max_own_len) {
  SharedPlan p;
  p.shared = plan_attention(groups, T, q_heads, kv_heads, D, max_group_len, max_shared_len);
  p.own = plan_attention(B, T, q_heads, kv_heads, D, max_q_len, max_own_len);
  p.own.first_part = p.shared.num_splits;
  const size_t rows = size_t(T) * q_heads, parts = size_t(p.shared.num_splits) + p.own.num_splits;
  const size_t ml = (parts * rows * sizeof(float2) + 255) / 256 * 256;
  p.own.ml_bytes = p.shared.ml_bytes = ml;
  p.bytes = ml + parts * rows * D * sizeof(float);
  return p;
}

hipError_t launch_shared(const AttnArgs& a, const SharedPlan& p, int cache_dtype, hipStream_t stream) {
  launch_part<Part::kShared>(a, p.shared, cache_dtype, stream);
  launch_part<Part::kOwn>(a, p.own, cache_dtype, stream);
  if (p.own.row_tile == 16)
    launch_join_shared<16, kBlock>(a, p, stream);
  else if (p.own.row_tile == 32)
    launch_join_shared<32, kBlock>(a, p, stream);
  else
    launch_join_shared<kManyRows, kTile>(a, p, stream);
  return hipGetLastError();
}

}  // namespace sv
