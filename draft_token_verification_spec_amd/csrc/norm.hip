// Norms of query and key heads with their rotary positions in the same pass,
// the gradients of that, and the append of normed keys to a paged cache.
//
// A head's row x of D channels becomes r R(t) (x w), r = (mean x^2 + eps)^-1/2,
// R the rotation by the row's angles (rope.hip): r is needed last, while the
// loads and the sum over the row are still on their way, and the first product
// is exact for bf16 rows and weights.  From the gradient dy with respect to it,
// with g = R^T dy,
//   dx = r (g w - x r (r mean(g w x))),   dw = sum over rows and heads of g x r,
// whose two sums over the row (of squares, of g w x) do not wait for each other;
// x is read again rather than r kept, which would be another array for the
// caller to hold and saves nothing of the bytes.
//
// Lanes and channels as in rope.hip: a group of 8, 16 or 32 lanes has a head's
// row in registers, 8 channels a lane; sums over the group are additions of
// lanes' neighbours and mirror images, which need no LDS.  A group asks for its
// next head's channels before it works on the present one's.
//
// The weights' gradients are summed by a thread over its heads and rows, by the
// workgroup in LDS, and by a second kernel over the workgroups, each in a fixed
// order.
//
// Measured: 64 rows of 32 + 8 heads of 128 bf16 channels 5.4 us (latency: a
// launch, the position, the angles); gradients of 8191 such rows, 252 MB in 52 +
// 5 us (4.8 TB/s; a plain copy reaches 5.1; their 28.7 million wave instructions
// alone take 47 us).
#include "sv_rope.hpp"

namespace sv {

namespace {

// ---------------------------------------------------------------------------
// rows of 8 channels a lane
// ---------------------------------------------------------------------------

// The sum over a group of 2^LG lanes, in each of them: neighbours, pairs, and
// then mirror images in 8 and in 16 lanes, whose halves hold the same by then.
template <int CTRL>
__device__ __forceinline__ float from_lane(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
template <int CTRL>
__device__ __forceinline__ double from_lane(double x) {
  const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(x), CTRL, 0xf, 0xf, true);
  const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(x), CTRL, 0xf, 0xf, true);
  return __hiloint2double(hi, lo);
}
__device__ __forceinline__ float from_other_row(float x) { return __shfl_xor(x, 16, 64); }
__device__ __forceinline__ double from_other_row(double x) { return __shfl_xor(x, 16, 64); }

template <int LG, typename F, typename Op>
__device__ __forceinline__ F over_group(F x, Op op) {
  x = op(x, from_lane<0xB1>(x));
  x = op(x, from_lane<0x4E>(x));
  x = op(x, from_lane<0x141>(x));
  if (LG >= 4) x = op(x, from_lane<0x140>(x));
  if (LG >= 5) x = op(x, from_other_row(x));
  return x;
}
template <int LG, typename F>
__device__ __forceinline__ F group_sum(F x) {
  return over_group<LG>(x, [](F a, F b) { return a + b; });
}

// A lane's place in its head: channels e0 .. e0 + 7, and what they are paired
// with.
struct Lane {
  int e0, D, rotary, half;
  bool live;         // the row has these channels
  bool interleaved;
};
template <int LG>
__device__ __forceinline__ Lane lane_of(int D, int rotary, int layout) {
  Lane l;
  l.e0 = (threadIdx.x & ((1 << LG) - 1)) * 8;
  l.D = D, l.rotary = rotary, l.half = rotary >> 1;
  l.live = l.e0 < D;
  l.interleaved = layout == SV_ROPE_INTERLEAVED;
  return l;
}
__device__ __forceinline__ bool is_first(const Lane& l, int e) { return l.interleaved ? (e & 1) == 0 : e < l.half; }
__device__ __forceinline__ int paired(const Lane& l, int e) {
  return e >= l.rotary ? e : l.interleaved ? e ^ 1 : e < l.half ? e + l.half : e - l.half;
}
__device__ __forceinline__ int angle_of(const Lane& l, int e) { return l.interleaved ? e >> 1 : e < l.half ? e : e - l.half; }

// Where LDS has the e-th angle and the weight of channel e.  VEC: what a lane
// reads in 16 bytes lies next to what its neighbours read along with it.
template <bool VEC>
__device__ __forceinline__ int angle_slot(const Lane& l, int e) {
  if (!VEC) return e;
  return l.interleaved ? ((e >> 1 & 1) * (l.half >> 2) + (e >> 2)) * 2 + (e & 1)
                       : ((e >> 1 & 3) * (l.half >> 3) + (e >> 3)) * 2 + (e & 1);
}
__device__ __forceinline__ int weight_slot(int e) {
  return (e >> 2 & 1) * (SV_ATTN_MAX_HEAD_DIM / 2) + (e >> 3) * 4 + (e & 3);
}

// A lane's 8 channels of a row as they are asked for, and as floats.  VEC: rows
// are 16-byte aligned, and heads and turned channels come in whole groups of 8;
// a lane beyond the row asks for its last channels.  (Interleaved pairs lie in
// the lane itself: asking for them does nothing.)
template <bool VEC, typename ET>
struct Channels {
  uint4 w[sizeof(ET) / 2];
  __device__ __forceinline__ void ask(const ET* row, const Lane& l, bool pairs) {
    if (pairs && l.interleaved) return;
    const int e = min(l.e0, l.D - 8);
    const uint4* p = reinterpret_cast<const uint4*>(row + (pairs ? paired(l, e) : e));
#pragma unroll
    for (int i = 0; i < int(sizeof(ET) / 2); ++i) w[i] = p[i];
  }
  __device__ __forceinline__ void get(const Lane& l, float (&x)[8]) const {
    if (sizeof(ET) == 2) {
      x[0] = bf16_lo(w[0].x), x[1] = bf16_hi(w[0].x), x[2] = bf16_lo(w[0].y), x[3] = bf16_hi(w[0].y);
      x[4] = bf16_lo(w[0].z), x[5] = bf16_hi(w[0].z), x[6] = bf16_lo(w[0].w), x[7] = bf16_hi(w[0].w);
    } else {
      const uint4 b = w[sizeof(ET) / 2 - 1];
      x[0] = __uint_as_float(w[0].x), x[1] = __uint_as_float(w[0].y), x[2] = __uint_as_float(w[0].z);
      x[3] = __uint_as_float(w[0].w), x[4] = __uint_as_float(b.x), x[5] = __uint_as_float(b.y);
      x[6] = __uint_as_float(b.z), x[7] = __uint_as_float(b.w);
    }
    if (!l.live) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.f;
    }
  }
};
template <typename ET>
struct Channels<false, ET> {
  float v[8];
  __device__ __forceinline__ void ask(const ET* row, const Lane& l, bool pairs) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = l.e0 + j;
      v[j] = e < l.D ? load1(row + (pairs ? paired(l, e) : e)) : 0.f;
    }
  }
  __device__ __forceinline__ void get(const Lane&, float (&x)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = v[j];
  }
};

// y turned: z holds what its channels are paired with (VEC and interleaved: y
// itself does).  (Explicitly fused, so that a row's bits do not depend on its
// alignment.)
template <bool VEC, typename F, typename F2>
__device__ __forceinline__ void turn8(F (&y)[8], const F (&z)[8], const Lane& l, const F2* cs) {
  if (!VEC) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = l.e0 + j;
      if (e >= l.rotary) continue;
      const F2 t = cs[angle_of(l, e)];
      y[j] = fma(y[j], t.x, is_first(l, e) ? -(z[j] * t.y) : z[j] * t.y);
    }
  } else if (l.e0 < l.rotary) {
    if (l.interleaved) {
      const F2* at = cs + (l.e0 >> 3) * 2;
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const F2 t = at[(j >> 2) * (l.half >> 2) * 2 + (j >> 1 & 1)];
        const F a = y[j], c = y[j + 1];
        y[j] = fma(a, t.x, -(c * t.y));
        y[j + 1] = fma(c, t.x, a * t.y);
      }
    } else {
      const bool first = l.e0 < l.half;
      const F2* at = cs + ((first ? l.e0 : l.e0 - l.half) >> 3) * 2;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const F2 t = at[(j >> 1) * (l.half >> 3) * 2 + (j & 1)];
        y[j] = fma(y[j], t.x, first ? -(z[j] * t.y) : z[j] * t.y);
      }
    }
  }
}

// The weights of queries' and keys' norms, to LDS as floats (none: ones), by the
// whole workgroup; zeros up to a whole number of lanes.
typedef float Weights[2][SV_ATTN_MAX_HEAD_DIM];
__device__ __forceinline__ void stage_weights(Weights& w, const NormWeights& n, int D) {
#pragma unroll
  for (int k = 0; k < 2; ++k)
    for (int e = threadIdx.x; e < SV_ATTN_MAX_HEAD_DIM; e += kRopeThreads) {
      const void* p = k ? n.k : n.q;
      float x = e < D ? 1.f : 0.f;
      if (p && e < D)
        x = n.dtype == SV_BF16 ? load1(static_cast<const uint16_t*>(p) + e) : load1(static_cast<const float*>(p) + e);
      w[k][weight_slot(e)] = x;
    }
}

template <bool VEC, typename F>
__device__ __forceinline__ void times_weights(F (&y)[8], const Lane& l, const float* w, bool pairs) {
  if (VEC) {
  const int e = pairs ? paired(l, l.e0) : l.e0;
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] *= w[weight_slot(e) + (j >> 2) * (SV_ATTN_MAX_HEAD_DIM / 2) + (j & 3)];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] *= w[weight_slot(pairs && l.e0 + j < l.D ? paired(l, l.e0 + j) : l.e0 + j)];
  }
}

// m^-1/2: the hardware's estimate and one step of Newton's method in binary64,
// so that the result adds no more than its own rounding to the sum's.
__device__ __forceinline__ double inverse_root(double m) {
  const double r = __builtin_amdgcn_rsqf(float(m));
  return r * (1.5 - 0.5 * m * r * r);
}

// The squares of a row's 8 channels, added pairwise.
__device__ __forceinline__ float squares(const float (&y)[8]) {
  const auto two = [&](int j) { return fmaf(y[j], y[j], y[j + 1] * y[j + 1]); };
  return (two(0) + two(2)) + (two(4) + two(6));
}

// y (and z, what it is paired with): normed and turned.
template <int LG, bool VEC>
__device__ __forceinline__ void norm_and_turn8(float (&y)[8], float (&z)[8], const Lane& l, const float2* cs,
                                               const float* w, const NormWeights& n) {
  const float r = float(inverse_root(double(group_sum<LG>(squares(y))) * n.inv_dim + n.eps));
  times_weights<VEC>(y, l, w, false);
  if (!VEC || !l.interleaved) times_weights<VEC>(z, l, w, true);
  turn8<VEC>(y, z, l, cs);
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] *= r;
}

// ---------------------------------------------------------------------------
// queries and keys, and gradients
// ---------------------------------------------------------------------------

// A group's items: the heads of a workgroup's rows in turn.
struct Item {
  int row, head;
  __device__ __forceinline__ void settle(int total) {
    while (head >= total) head -= total, ++row;
  }
};

// mscale * (cos, sin) of the angles of rows t0 .. t0 + rows - 1.
template <int ROWS, bool VEC>
__device__ __forceinline__ void angles_of_rows(float2 (*cs)[kMaxPairs], const NormRopeArgs& a, const Lane& l, int t0,
                                               int rows, float sign) {
  const int pairs = l.half;
  for (int i = threadIdx.x; i < ROWS * pairs; i += kRopeThreads) {
    const int r = ROWS == 1 ? 0 : i / pairs, e = i - r * pairs;
    if (r < rows) cs[r][angle_slot<VEC>(l, e)] = turn_of(double(a.positions[t0 + r]), a.freq[e], a.mscale, sign);
  }
}

// One of two arrays of rows, by value: a reference to either would be a load
// through an address.
template <typename Rows>
__device__ __forceinline__ Rows one_of(bool second, const Rows& a, const Rows& b) {
  return {second ? b.p : a.p, second ? b.token : a.token, second ? b.head : a.head};
}

template <typename ET, typename Rows>
__device__ __forceinline__ auto row_of(const NormRopeArgs& a, const Rows& q, const Rows& k, int t0, const Item& it) {
  const bool key = it.head >= a.q_heads;
  const Rows x = one_of(key, q, k);
  return static_cast<ET*>(x.p) + int64_t(t0 + it.row) * x.token + int64_t(key ? it.head - a.q_heads : it.head) * x.head;
}

template <int LG, int ROWS, bool VEC, typename ET>
__global__ __launch_bounds__(kRopeThreads) void norm_rope_kernel(NormRopeArgs a) {
  __shared__ __align__(16) float2 cs[ROWS][kMaxPairs];
  __shared__ __align__(16) Weights w;
  const int t0 = blockIdx.x * ROWS, rows = min(ROWS, a.T - t0);
  const Lane l = lane_of<LG>(a.D, a.rotary, a.layout);
  const int total = a.q_heads + a.k_heads;
  Item it = {0, int(threadIdx.x >> LG)};
  it.settle(total);
  Channels<VEC, ET> y0, z0;
  if (it.row < rows) {
    const ET* x = row_of<const ET>(a, a.q, a.k, t0, it);
    y0.ask(x, l, false);
    z0.ask(x, l, true);
  }
  stage_weights(w, a.norm, a.D);
  angles_of_rows<ROWS, VEC>(cs, a, l, t0, rows, 1.f);
  __syncthreads();
  while (it.row < rows) {
    float y[8], z[8];
    y0.get(l, y);
    z0.get(l, z);
    Item next = {it.row, it.head + (kRopeThreads >> LG)};
    next.settle(total);
    {
      const ET* x = row_of<const ET>(a, a.q, a.k, t0, next.row < rows ? next : it);
      y0.ask(x, l, false);
      z0.ask(x, l, true);
    }
    norm_and_turn8<LG, VEC>(y, z, l, cs[it.row], w[it.head >= a.q_heads], a.norm);
    if (l.live) put8<VEC>(row_of<ET>(a, a.q_out, a.k_out, t0, it), l.e0, a.D, y);
    it = next;
  }
}

constexpr int kMostParts = 1024;  // workgroups of the backward pass: 16 waves a compute unit

template <int LG, int ROWS, bool VEC, typename ET>
__global__ __launch_bounds__(kRopeThreads) void norm_rope_backward_kernel(NormRopeArgs a) {
  __shared__ __align__(16) float2 cs[2][ROWS][kMaxPairs];
  __shared__ __align__(16) Weights w;
  __shared__ float sums[kRopeThreads / 64][2][8 << LG];
  const Lane l = lane_of<LG>(a.D, a.rotary, a.layout);
  const int total = a.q_heads + a.k_heads;
  const float inv_dim = float(a.norm.inv_dim);
  float dw[2][8] = {};
  stage_weights(w, a.norm, a.D);
  int buf = 0;
  // (the barrier of some rows ends every read of the angles of those before)
  for (int t0 = blockIdx.x * ROWS; t0 < a.T; t0 += gridDim.x * ROWS, buf ^= 1) {
    const int rows = min(ROWS, a.T - t0);
    Item it = {0, int(threadIdx.x >> LG)};
    it.settle(total);
    Channels<VEC, ET> x0, g0, z0;
    const auto ask = [&](const Item& i) {
      const ET* dy = row_of<const ET>(a, a.dq, a.dk, t0, i);
      x0.ask(row_of<const ET>(a, a.q, a.k, t0, i), l, false);
      g0.ask(dy, l, false);
      z0.ask(dy, l, true);
    };
    if (it.row < rows) ask(it);
    angles_of_rows<ROWS, VEC>(cs[buf], a, l, t0, rows, -1.f);
    __syncthreads();
    while (it.row < rows) {
      float x[8], g[8], z[8];
      x0.get(l, x);
      g0.get(l, g);
      z0.get(l, z);
      Item next = {it.row, it.head + (kRopeThreads >> LG)};
      next.settle(total);
      ask(next.row < rows ? next : it);
      turn8<VEC>(g, z, l, cs[buf][it.row]);
      const bool key = it.head >= a.q_heads;
      const float r = float(inverse_root(double(group_sum<LG>(squares(x))) * a.norm.inv_dim + a.norm.eps));
      float dot = 0.f, y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = g[j];
      times_weights<VEC>(y, l, w[key], false);
#pragma unroll
      for (int j = 0; j < 8; ++j) dot = fmaf(y[j], x[j], dot);
      const float c = group_sum<LG>(dot) * r * inv_dim;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] *= r;
        if (key)
          dw[1][j] = fmaf(g[j], x[j], dw[1][j]);
        else
          dw[0][j] = fmaf(g[j], x[j], dw[0][j]);
        y[j] = r * fmaf(-x[j], c, y[j]);
      }
      if (l.live) put8<VEC>(row_of<ET>(a, a.q_out, a.k_out, t0, it), l.e0, a.D, y);
      it = next;
    }
  }
  if (!a.part) return;
  // the wave's groups, then the waves
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float x = dw[k][j];
#pragma unroll
      for (int o = 32; o >= 1 << LG; o >>= 1) x += __shfl_xor(x, o, 64);
      if ((threadIdx.x & 63) < 1 << LG) sums[threadIdx.x >> 6][k][l.e0 + j] = x;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.D; i += kRopeThreads) {
    const int k = i >= a.D, e = k ? i - a.D : i;
    float x = 0.f;
#pragma unroll
    for (int v = 0; v < kRopeThreads / 64; ++v) x += sums[v][k][e];
    a.part[int64_t(blockIdx.x) * (2 * a.D) + i] = x;
  }
}

// 16 channels a workgroup, 64 threads a channel.
constexpr int kJoinThreads = 1024;
__global__ __launch_bounds__(kJoinThreads) void weight_gradient_kernel(NormRopeArgs a, int parts) {
  __shared__ float sums[kJoinThreads];
  const int i = blockIdx.x * 16 + (threadIdx.x & 15);
  float x = 0.f;
  if (i < 2 * a.D) {
#pragma unroll 8
    for (int p = threadIdx.x >> 4; p < parts; p += kJoinThreads / 16) x += a.part[int64_t(p) * (2 * a.D) + i];
  }
  sums[threadIdx.x] = x;
  for (int n = kJoinThreads / 2; n >= 16; n >>= 1) {
    __syncthreads();
    if (threadIdx.x < n) sums[threadIdx.x] += sums[threadIdx.x + n];
  }
  if (threadIdx.x >= 16 || i >= 2 * a.D) return;
  float* out = i < a.D ? a.dq_weight : a.dk_weight;
  if (out) out[i < a.D ? i : i - a.D] = sums[threadIdx.x];
}

// ---------------------------------------------------------------------------
// into a cache
// ---------------------------------------------------------------------------

// A number that rounds to e4m3 as x does: x without what binary32 has no place
// for, its last bit set where something is missing.  (Beyond binary32's normal
// numbers: the nearest one.)
__device__ __forceinline__ float shortened(double x) {
  const uint64_t bits = __double_as_longlong(x);
  const uint32_t high = uint32_t(bits >> 32), low = uint32_t(bits);
  const uint32_t size = high & 0x7fffffffu;
  if (size - (897u << 20) >= 253u << 20) return float(x);
  return __uint_as_float((high & 0x80000000u) | ((size - (896u << 20)) << 3) | (low >> 29) | ((low & 0x1fffffffu) != 0));
}

// y (and z) normed and turned in binary64: keys, which are stored once and read
// by every later row, are so the nearest 8-bit values (FP8; in binary32 some
// 10^-6 of them are not), or the nearest binary32 ones on their way to bf16, for
// finite rows of any size.  The root is the hardware's binary64 estimate (some
// 2^-24 off) and one step of Newton's method.
template <int LG, bool VEC, bool FP8>
__device__ __forceinline__ void norm_and_turn_key8(float (&y)[8], const float (&z)[8], const Lane& l, const double2* cs,
                                                   const float* w, const NormWeights& n) {
  double u[8], v[8], sq = 0.;
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] = y[j], sq = fma(u[j], u[j], sq);
  const double m = group_sum<LG>(sq) * n.inv_dim + n.eps;
  double r = __builtin_amdgcn_rsq(m);  // (the squares of binary32's larger numbers are beyond its range)
  r *= 1.5 - 0.5 * m * r * r;
  times_weights<VEC>(u, l, w, false);
  if (!VEC || !l.interleaved) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = z[j];
    times_weights<VEC>(v, l, w, true);
  }
  turn8<VEC>(u, v, l, cs);
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = FP8 ? shortened(u[j] * r) : float(u[j] * r);
}

// One workgroup per row, as rope.hip's append.  Bound by HBM for many rows: 8285
// binary32 rows of 32 + 8 + 8 heads of 128 into an 8-bit cache, 357 MB in 75 us
// (4.8 TB/s); by latency for few: 1280 bf16 rows of the same heads 11.5 us.  Four
// rows a workgroup, or a head's channels asked for ahead, cost registers and so
// waves (85 to 98 us, 13 to 16).  Vector rows are held to the 96 registers of five
// waves a SIMD, for which up to five are spilled, of a key's binary64 channels.
// A row's angles, weights and barriers are the same for few heads: 8192 rows of 8 +
// 1 + 1 heads take 29 us a call for 42 MB, 32768 of 4 + 1 + 1 82 for 101.
template <int LG, bool VEC, bool FP8, typename ET>
__global__ __launch_bounds__(kRopeThreads, VEC ? 5 : 4) void append_normed_kernel(AppendArgs a) {
  __shared__ __align__(16) float2 cs[kMaxPairs];
  __shared__ double2 exact[kMaxPairs];
  __shared__ __align__(16) Weights w;
  const PagedView& cache = a.cache;
  const int t = blockIdx.x, heads = cache.heads;
  // requests of equally many rows are found at once, others by a search
  int b = int(int64_t(t) * a.B / a.T);
  int end = a.query_start[b + 1];
  if (t < a.query_start[b] || t >= end) {
    b = find_sequence(a.query_start, a.B, t, threadIdx.x & 63);
    if (b < 0) return;
    end = a.query_start[b + 1];
    if (t >= end) return;  // behind the last request
  }
  const int place = max(a.kv_len[b], 0) - (end - t);
  const int page = page_of(cache, b, place);
  const double position = a.positions ? double(a.positions[t]) : double(place);
  const Lane l = lane_of<LG>(cache.D, a.rotary, a.layout);
  stage_weights(w, a.norm, cache.D);
  for (int i = threadIdx.x; i < l.half; i += kRopeThreads) {
    double s, c;
    sincospi(half_turns(position, a.freq[i]), &s, &c);
    const int at = angle_slot<VEC>(l, i);
    exact[at] = make_double2(c * a.mscale, s * a.mscale);
    cs[at] = make_float2(float(c * a.mscale), float(s * a.mscale));
  }
  __syncthreads();

  const int slot = place & ((1 << cache.page_shift) - 1);
  const int total = a.q_heads + (page >= 0 ? 2 * heads : 0);
  for (int i = threadIdx.x >> LG; i < total; i += kRopeThreads >> LG) {
    Channels<VEC, ET> y0, z0;
    float y[8], z[8];
    if (i < a.q_heads) {
      const ET* x = static_cast<const ET*>(a.q.p) + int64_t(t) * a.q.token + i * a.q.head;
      y0.ask(x, l, false);
      z0.ask(x, l, true);
      y0.get(l, y);
      z0.get(l, z);
      norm_and_turn8<LG, VEC>(y, z, l, cs, w[0], a.norm);
      if (l.live) put8<VEC>(static_cast<ET*>(a.q_out.p) + int64_t(t) * a.q_out.token + i * a.q_out.head, l.e0, l.D, y);
    } else if (i < a.q_heads + heads) {
      const int h = i - a.q_heads;
      const ET* x = static_cast<const ET*>(a.k.p) + int64_t(t) * a.k.token + h * a.k.head;
      y0.ask(x, l, false);
      z0.ask(x, l, true);
      y0.get(l, y);
      z0.get(l, z);
      norm_and_turn_key8<LG, VEC, FP8>(y, z, l, exact, w[1], a.norm);
      put_cache<FP8>(cache, cache.k, page * cache.k_page + slot * cache.k_token + h * cache.k_head, cache.k_scale,
                     ((int64_t(page) * heads + h) << cache.page_shift) + slot, l.e0, l.live, y, 1 << LG);
    } else {
      const int h = i - a.q_heads - heads;
      y0.ask(static_cast<const ET*>(a.v.p) + int64_t(t) * a.v.token + h * a.v.head, l, false);
      y0.get(l, y);
      put_cache<FP8>(cache, cache.v, page * cache.v_page + slot * cache.v_token + h * cache.v_head, cache.v_scale,
                     ((int64_t(page) * heads + h) << cache.page_shift) + slot, l.e0, l.live, y, 1 << LG);
    }
  }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

bool vec_of(const NormRopeArgs& a, int elem, bool backward) {
  bool vec = channels_vec(a.D, a.rotary, a.layout);
  if (a.q_heads > 0)
    vec = vec && rows_vec(a.q.p, a.q.token, a.q.head, elem) && rows_vec(a.q_out.p, a.q_out.token, a.q_out.head, elem) &&
          (!backward || rows_vec(a.dq.p, a.dq.token, a.dq.head, elem));
  if (a.k_heads > 0)
    vec = vec && rows_vec(a.k.p, a.k.token, a.k.head, elem) && rows_vec(a.k_out.p, a.k_out.token, a.k_out.head, elem) &&
          (!backward || rows_vec(a.dk.p, a.dk.token, a.dk.head, elem));
  return vec;
}

// Rows that a workgroup takes at a time: several where there are enough to fill
// the card with, whose angles then keep all threads busy and whose heads divide
// into whole turns of its groups (bf16, 40 heads of 128, whole calls: 8191 rows'
// gradients 66 us one row at a time and 57 four, 16000 rows 81 and 69; of 64
// channels 46 and 35; below 4000 rows no difference).
constexpr int kManyRowsAtATime = 4;
bool many(int T) { return T >= 1024 * kManyRowsAtATime; }

template <int LG, int ROWS, bool VEC, typename ET>
void launch_rows_of(const NormRopeArgs& a, bool backward, hipStream_t stream) {
  const int blocks = (a.T + ROWS - 1) / ROWS;
  if (backward)
    hipLaunchKernelGGL((norm_rope_backward_kernel<LG, ROWS, VEC, ET>), dim3(norm_parts(a.T)), dim3(kRopeThreads), 0,
                       stream, a);
  else
    hipLaunchKernelGGL((norm_rope_kernel<LG, ROWS, VEC, ET>), dim3(blocks), dim3(kRopeThreads), 0, stream, a);
}

template <int LG, bool VEC, typename ET>
void launch_heads(const NormRopeArgs& a, bool backward, hipStream_t stream) {
  many(a.T) ? launch_rows_of<LG, kManyRowsAtATime, VEC, ET>(a, backward, stream)
            : launch_rows_of<LG, 1, VEC, ET>(a, backward, stream);
}

template <bool VEC, typename ET>
void launch_type(const NormRopeArgs& a, bool backward, hipStream_t stream) {
  const int lg = head_lanes_log2(a.D);
  lg == 3   ? launch_heads<3, VEC, ET>(a, backward, stream)
  : lg == 4 ? launch_heads<4, VEC, ET>(a, backward, stream)
            : launch_heads<5, VEC, ET>(a, backward, stream);
}

void launch_of(const NormRopeArgs& a, int dtype, bool backward, hipStream_t stream) {
  const bool vec = vec_of(a, dtype == SV_BF16 ? 2 : 4, backward);
  if (dtype == SV_BF16)
    vec ? launch_type<true, uint16_t>(a, backward, stream) : launch_type<false, uint16_t>(a, backward, stream);
  else
    vec ? launch_type<true, float>(a, backward, stream) : launch_type<false, float>(a, backward, stream);
}

template <bool VEC, bool FP8, typename ET>
void launch_append_type(const AppendArgs& a, hipStream_t stream) {
  const dim3 grid(a.T), block(kRopeThreads);
  const int lg = head_lanes_log2(a.cache.D);
  if (lg == 3)
    hipLaunchKernelGGL((append_normed_kernel<3, VEC, FP8, ET>), grid, block, 0, stream, a);
  else if (lg == 4)
    hipLaunchKernelGGL((append_normed_kernel<4, VEC, FP8, ET>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((append_normed_kernel<5, VEC, FP8, ET>), grid, block, 0, stream, a);
}

template <bool VEC, bool FP8>
void launch_append_of(const AppendArgs& a, int dtype, hipStream_t stream) {
  dtype == SV_BF16 ? launch_append_type<VEC, FP8, uint16_t>(a, stream) : launch_append_type<VEC, FP8, float>(a, stream);
}

}  // namespace

int norm_parts(int T) {
  const int blocks = many(T) ? (T + kManyRowsAtATime - 1) / kManyRowsAtATime : T;
  return blocks < kMostParts ? blocks : kMostParts;
}

hipError_t launch_norm(const NormRopeArgs& a, int dtype, hipStream_t stream) {
  launch_of(a, dtype, false, stream);
  return hipGetLastError();
}

hipError_t launch_norm_backward(const NormRopeArgs& a, int dtype, hipStream_t stream) {
  if (a.T > 0) launch_of(a, dtype, true, stream);
  if (a.dq_weight || a.dk_weight)
    hipLaunchKernelGGL(weight_gradient_kernel, dim3((2 * a.D + 15) / 16), dim3(kJoinThreads), 0, stream, a, norm_parts(a.T));
  return hipGetLastError();
}

hipError_t launch_append_normed(const AppendArgs& a, int dtype, int cache_dtype, hipStream_t stream) {
  const int elem = dtype == SV_BF16 ? 2 : 4;
  bool vec = channels_vec(a.cache.D, a.rotary, a.layout) && rows_vec(a.k.p, a.k.token, a.k.head, elem) &&
             rows_vec(a.v.p, a.v.token, a.v.head, elem);
  if (a.q_heads > 0)
    vec = vec && rows_vec(a.q.p, a.q.token, a.q.head, elem) && rows_vec(a.q_out.p, a.q_out.token, a.q_out.head, elem);
  if (cache_dtype == SV_E4M3)
    vec ? launch_append_of<true, true>(a, dtype, stream) : launch_append_of<false, true>(a, dtype, stream);
  else
    vec ? launch_append_of<true, false>(a, dtype, stream) : launch_append_of<false, false>(a, dtype, stream);
  return hipGetLastError();
}

}  // namespace sv
