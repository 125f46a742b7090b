// Norms of query and key heads with their rotary positions in the same pass,
// and the gradients of that.
//
// A head's row x of D channels becomes R(t) (x r w), r = (mean x^2 + eps)^-1/2,
// R the rotation by the row's angles (rope.hip).  From the gradient dy with
// respect to it, with g = R^T dy and u = x r,
//   dx = r (g w - u mean(g w u)),   dw = sum over rows and heads of g u:
// x is read again rather than r kept, which would be another array for the
// caller to hold and saves nothing of the bytes.
//
// Lanes and channels as in rope.hip: a group of 8, 16 or 32 lanes has a head's
// row in registers, so the two means are reductions over the group.
// The weights' gradients are summed by a thread over its heads and rows, by the
// workgroup in LDS, and by a second kernel over the workgroups, each in a fixed
// order.
#include "sv_rope.hpp"

namespace sv {

namespace {

// A thread's items, heads of a workgroup's rows in turn: the i-th of the
// workgroup's groups starts at the i-th.
struct Item {
  int row, head;
  __device__ __forceinline__ void settle(int total) {
    while (head >= total) head -= total, ++row;
  }
};

// mscale * (cos, sin) of the angles of rows t0 .. t0 + rows - 1.
template <int ROWS>
__device__ __forceinline__ void angles_of_rows(float2 (*cs)[kMaxPairs], const NormRopeArgs& a, int t0, int rows, float sign) {
  const int pairs = a.rotary >> 1;
  for (int i = threadIdx.x; i < ROWS * pairs; i += kRopeThreads) {
    const int r = ROWS == 1 ? 0 : i / pairs, e = i - r * pairs;
    if (r < rows) cs[r][e] = turn_of(double(a.positions[t0 + r]), a.freq[e], a.mscale, sign);
  }
}

template <int ROWS, bool VEC, typename ET>
__global__ __launch_bounds__(kRopeThreads) void norm_rope_kernel(NormRopeArgs a) {
  __shared__ float2 cs[ROWS][kMaxPairs];
  __shared__ float w[2][SV_ATTN_MAX_HEAD_DIM];
  const int t0 = blockIdx.x * ROWS, rows = min(ROWS, a.T - t0);
  stage_weights(w, a.norm, a.D);
  angles_of_rows<ROWS>(cs, a, t0, rows, 1.f);
  __syncthreads();
  const int lg = head_lanes_log2(a.D), lanes = 1 << lg;
  const int e0 = (threadIdx.x & (lanes - 1)) * 8;
  const int total = a.q_heads + a.k_heads;
  Item it = {0, int(threadIdx.x >> lg)};
  for (it.settle(total); it.row < rows; it.head += kRopeThreads >> lg, it.settle(total)) {
    const bool key = it.head >= a.q_heads;
    const int h = key ? it.head - a.q_heads : it.head;
    const RowsIn& in = key ? a.k : a.q;
    const RowsOut& out = key ? a.k_out : a.q_out;
    const int64_t t = t0 + it.row;
    float y[8] = {};
    normed8<VEC>(static_cast<const ET*>(in.p) + t * in.token + h * in.head, e0, a.D, a.rotary, a.layout, cs[it.row],
                 w[key], a.norm, lanes, y);
    if (e0 < a.D) put8<VEC>(static_cast<ET*>(out.p) + t * out.token + h * out.head, e0, a.D, y);
  }
}

constexpr int kMostParts = 1024;  // workgroups of the backward pass: 16 waves a compute unit

template <int ROWS, bool VEC, typename ET>
__global__ __launch_bounds__(kRopeThreads) void norm_rope_backward_kernel(NormRopeArgs a) {
  __shared__ float2 cs[2][ROWS][kMaxPairs];
  __shared__ float w[2][SV_ATTN_MAX_HEAD_DIM];
  __shared__ float sums[kRopeThreads / 64][2][SV_ATTN_MAX_HEAD_DIM];
  const int lg = head_lanes_log2(a.D), lanes = 1 << lg;
  const int e0 = (threadIdx.x & (lanes - 1)) * 8;
  const int total = a.q_heads + a.k_heads;
  const float inv_dim = float(a.norm.inv_dim);
  float dw[2][8] = {};
  stage_weights(w, a.norm, a.D);
  int buf = 0;
  // (the barrier of some rows ends every read of the angles of those before)
  for (int t0 = blockIdx.x * ROWS; t0 < a.T; t0 += gridDim.x * ROWS, buf ^= 1) {
    const int rows = min(ROWS, a.T - t0);
    angles_of_rows<ROWS>(cs[buf], a, t0, rows, -1.f);
    __syncthreads();
    Item it = {0, int(threadIdx.x >> lg)};
    for (it.settle(total); it.row < rows; it.head += kRopeThreads >> lg, it.settle(total)) {
      const bool key = it.head >= a.q_heads;
      const int h = key ? it.head - a.q_heads : it.head;
      const RowsIn& in = key ? a.k : a.q;
      const RowsIn& grad = key ? a.dk : a.dq;
      const RowsOut& out = key ? a.k_out : a.q_out;
      const int64_t t = t0 + it.row;
      const ET* px = static_cast<const ET*>(in.p) + t * in.token + h * in.head;
      const ET* pg = static_cast<const ET*>(grad.p) + t * grad.token + h * grad.head;
      float u[8] = {}, g[8] = {};
      load_pairs8<VEC>(px, e0, a.D, 0, a.layout, u, g);
      if (e0 < a.D) turned8<VEC>(pg, e0, a.D, a.rotary, a.layout, cs[buf][it.row], g);
      const float r = inverse_norm(u, a.norm, lanes);
      float dot = 0.f, y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[j] *= r;
        if (key)
          dw[1][j] = fmaf(g[j], u[j], dw[1][j]);
        else
          dw[0][j] = fmaf(g[j], u[j], dw[0][j]);
        y[j] = VEC || e0 + j < a.D ? g[j] * w[key][min(e0 + j, SV_ATTN_MAX_HEAD_DIM - 1)] : 0.f;
        dot = fmaf(y[j], u[j], dot);
      }
      const float c = group_sum(dot, lanes) * inv_dim;
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = r * (y[j] - u[j] * c);
      if (e0 < a.D) put8<VEC>(static_cast<ET*>(out.p) + t * out.token + h * out.head, e0, a.D, y);
    }
  }
  if (!a.part) return;
  // the wave's groups, then the waves
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float x = dw[k][j];
      for (int o = 32; o >= lanes; o >>= 1) x += __shfl_xor(x, o, 64);
      if ((threadIdx.x & 63) < lanes) sums[threadIdx.x >> 6][k][e0 + j] = x;
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
  if (i < 2 * a.D)
    for (int p = threadIdx.x >> 4; p < parts; p += kJoinThreads / 16) x += a.part[int64_t(p) * (2 * a.D) + i];
  sums[threadIdx.x] = x;
  for (int n = kJoinThreads / 2; n >= 16; n >>= 1) {
    __syncthreads();
    if (threadIdx.x < n) sums[threadIdx.x] += sums[threadIdx.x + n];
  }
  if (threadIdx.x >= 16 || i >= 2 * a.D) return;
  float* out = i < a.D ? a.dq_weight : a.dk_weight;
  if (out) out[i < a.D ? i : i - a.D] = sums[threadIdx.x];
}

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
// the card with.
constexpr int kManyRowsAtATime = 4;
bool many(int T) { return T >= 1024 * kManyRowsAtATime; }

template <int ROWS, bool VEC, typename ET>
void launch_rows_of(const NormRopeArgs& a, bool backward, hipStream_t stream) {
  const int blocks = (a.T + ROWS - 1) / ROWS;
  if (backward)
    hipLaunchKernelGGL((norm_rope_backward_kernel<ROWS, VEC, ET>), dim3(norm_parts(a.T)), dim3(kRopeThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((norm_rope_kernel<ROWS, VEC, ET>), dim3(blocks), dim3(kRopeThreads), 0, stream, a);
}

template <bool VEC, typename ET>
void launch_type(const NormRopeArgs& a, bool backward, hipStream_t stream) {
  many(a.T) ? launch_rows_of<kManyRowsAtATime, VEC, ET>(a, backward, stream) : launch_rows_of<1, VEC, ET>(a, backward, stream);
}

void launch_of(const NormRopeArgs& a, int dtype, bool backward, hipStream_t stream) {
  const bool vec = vec_of(a, dtype == SV_BF16 ? 2 : 4, backward);
  if (dtype == SV_BF16)
    vec ? launch_type<true, uint16_t>(a, backward, stream) : launch_type<false, uint16_t>(a, backward, stream);
  else
    vec ? launch_type<true, float>(a, backward, stream) : launch_type<false, float>(a, backward, stream);
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

}  // namespace sv
