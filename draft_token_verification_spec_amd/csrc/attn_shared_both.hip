// The shared and the own part of attention behind shared tokens in one launch
// (attn_shared.hip joins their parts).
//
// Those of the shared part, which take longer, come first.  (Eight of either kind
// in turn, which has both on every compute unit from the start, take as long or a
// little longer: 128 requests behind 8000 tokens 66 and 67 us, verification of 256
// behind 8 prompts 250 and 252.)
#include "sv_attn_kernels.hpp"
#include "sv_attn_shared.hpp"

namespace sv {

namespace {

// The place in a grid of (x, heads, splits) of its i-th workgroup.
__device__ __forceinline__ Block nth_block(uint32_t i, uint32_t nx, uint32_t heads) {
  const uint32_t row = i / nx;
  return {i - row * nx, row % heads, row / heads, nx};
}

template <int DP, int MT>
struct FewLds {
  __align__(16) FewValues<DP> values;
  FewStats<MT> stat_m, stat_l;
};
template <int DP>
struct ManyLds {
  __align__(16) ManyKeys<DP> keys;
  __align__(16) ManyValues<DP> values;
  __align__(16) ManyState state;
  __align__(16) ManyMarks marks;
};

// S, O: tiles of 16 rows of the shared and of the own part; S == 0: 128 rows.
template <int DP, bool FP8, int PAGES, int S, int O>
__global__ __launch_bounds__(kAttnThreads, DP > 64 ? 2 : 3) void shared_and_own_kernel(
    AttnArgs a, SharedPlan p, uint32_t shared_blocks) {
  constexpr int kSharedLds = S == 0 ? int(sizeof(ManyLds<DP>)) : int(sizeof(FewLds<DP, S ? S : 1>));
  constexpr int kOwnLds = int(sizeof(FewLds<DP, O>));
  __shared__ __align__(16) char lds[kSharedLds > kOwnLds ? kSharedLds : kOwnLds];
  // (either kind's number is rounded up to the XCDs', so that both are dealt to them alike)
  const bool own = blockIdx.x >= shared_blocks;
  const uint32_t i = own ? blockIdx.x - shared_blocks : blockIdx.x, heads = a.cache.heads;
  if (own) {
    const uint32_t nx = a.B * p.own.tiles;
    if (i >= nx * heads * p.own.num_splits) return;
    FewLds<DP, O>& s = *reinterpret_cast<FewLds<DP, O>*>(lds);
    few_rows<DP, O, FP8, false, Part::kOwn>(a, p.own, s.values, s.stat_m, s.stat_l, nth_block(i, nx, heads));
  } else {
    const uint32_t nx = a.groups * p.shared.tiles;
    if (i >= nx * heads * p.shared.num_splits) return;
    if constexpr (S == 0) {
      ManyLds<DP>& s = *reinterpret_cast<ManyLds<DP>*>(lds);
      many_rows<DP, FP8, PAGES, Part::kShared>(a, p.shared, s.keys, s.values, s.state, s.marks, nth_block(i, nx, heads));
    } else {
      FewLds<DP, S>& s = *reinterpret_cast<FewLds<DP, S>*>(lds);
      few_rows<DP, S, FP8, false, Part::kShared>(a, p.shared, s.values, s.stat_m, s.stat_l, nth_block(i, nx, heads));
    }
  }
}

template <int DP, bool FP8, int PAGES, int S, int O>
void launch_both(const AttnArgs& a, const SharedPlan& p, hipStream_t stream) {
  const auto blocks = [&](int64_t n, const AttnPlan& q) {
    return uint32_t((n * q.tiles * a.cache.heads * q.num_splits + 7) / 8 * 8);
  };
  const uint32_t shared = blocks(a.groups, p.shared), own = blocks(a.B, p.own);
  hipLaunchKernelGGL((shared_and_own_kernel<DP, FP8, PAGES, S, O>), dim3(shared + own), dim3(kAttnThreads), 0, stream, a, p,
                     shared);
}

template <int DP, bool FP8, int O>
void launch_tiles(const AttnArgs& a, const SharedPlan& p, hipStream_t stream) {
  if (p.shared.row_tile > 32)
    a.cache.page_shift < 6 ? launch_both<DP, FP8, 1, 0, O>(a, p, stream) : launch_both<DP, FP8, 2, 0, O>(a, p, stream);
  else if (O == 2 || p.shared.row_tile == 32)
    launch_both<DP, FP8, 1, 2, O>(a, p, stream);
  else
    launch_both<DP, FP8, 1, 1, 1>(a, p, stream);
}

template <int DP, bool FP8>
void launch_dp(const AttnArgs& a, const SharedPlan& p, hipStream_t stream) {
  p.own.row_tile == 16 ? launch_tiles<DP, FP8, 1>(a, p, stream) : launch_tiles<DP, FP8, 2>(a, p, stream);
}

}  // namespace

bool launch_shared_and_own(const AttnArgs& a, const SharedPlan& p, int cache_dtype, hipStream_t stream) {
  // heads of 256 channels fill the registers alone; requests of many rows are a
  // matter of the matrix units themselves; a token's page is looked up by its
  // lane only in the kernels of their own
  if (a.cache.D > 128 || p.own.row_tile > 32 || p.shared.row_tile < p.own.row_tile || looks_up_each_token(a.cache))
    return false;
  const auto blocks = [&](int64_t n, const AttnPlan& q) { return n * q.tiles * a.cache.heads * q.num_splits; };
  if (blocks(a.groups, p.shared) + blocks(a.B, p.own) > INT32_MAX / kAttnThreads) return false;
  if (cache_dtype == SV_E4M3)
    a.cache.D <= 64 ? launch_dp<64, true>(a, p, stream) : launch_dp<128, true>(a, p, stream);
  else
    a.cache.D <= 64 ? launch_dp<64, false>(a, p, stream) : launch_dp<128, false>(a, p, stream);
  return true;
}

}  // namespace sv
