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

template <bool VEC, typename ET>
__global__ __launch_bounds__(kRopeThreads) void norm_rope_kernel(NormRopeArgs a) {
  __shared__ float2 cs[kMaxPairs];
  __shared__ float w[2][SV_ATTN_MAX_HEAD_DIM];
  const int t = blockIdx.x;
  stage_weights(w, a.norm, a.D);
  make_angles(cs, a.freq, a.rotary >> 1, a.rotary ? double(a.positions[t]) : 0., a.mscale, 1.f);
  __syncthreads();
  const int lg = head_lanes_log2(a.D), lanes = 1 << lg;
  const int e0 = (threadIdx.x & (lanes - 1)) * 8;
  const int total = a.q_heads + a.k_heads;
  for (int g = threadIdx.x >> lg; g < total; g += kRopeThreads >> lg) {
    const bool key = g >= a.q_heads;
    const int h = key ? g - a.q_heads : g;
    const RowsIn& in = key ? a.k : a.q;
    const RowsOut& out = key ? a.k_out : a.q_out;
    float y[8] = {};
    normed8<VEC>(static_cast<const ET*>(in.p) + int64_t(t) * in.token + h * in.head, e0, a.D, a.rotary, a.layout, cs,
                 w[key], a.norm.eps, lanes, y);
    if (e0 < a.D) put8<VEC>(static_cast<ET*>(out.p) + int64_t(t) * out.token + h * out.head, e0, a.D, y);
  }
}

constexpr int kMostParts = 1024;  // workgroups of the backward pass: 16 waves a compute unit

template <bool VEC, typename ET>
__global__ __launch_bounds__(kRopeThreads) void norm_rope_backward_kernel(NormRopeArgs a) {
  __shared__ float2 cs[2][kMaxPairs];
  __shared__ float w[2][SV_ATTN_MAX_HEAD_DIM];
  __shared__ float sums[kRopeThreads / 64][2][SV_ATTN_MAX_HEAD_DIM];
  const int lg = head_lanes_log2(a.D), lanes = 1 << lg;
  const int e0 = (threadIdx.x & (lanes - 1)) * 8;
  const int total = a.q_heads + a.k_heads;
  float dw[2][8] = {};
  stage_weights(w, a.norm, a.D);
  int buf = 0;
  // (the barrier of a row ends every read of the angles of the row before)
  for (int t = blockIdx.x; t < a.T; t += gridDim.x, buf ^= 1) {
    make_angles(cs[buf], a.freq, a.rotary >> 1, a.rotary ? double(a.positions[t]) : 0., a.mscale, -1.f);
    __syncthreads();
    for (int i = threadIdx.x >> lg; i < total; i += kRopeThreads >> lg) {
      const bool key = i >= a.q_heads;
      const int h = key ? i - a.q_heads : i;
      const RowsIn& in = key ? a.k : a.q;
      const RowsIn& grad = key ? a.dk : a.dq;
      const RowsOut& out = key ? a.k_out : a.q_out;
      const ET* px = static_cast<const ET*>(in.p) + int64_t(t) * in.token + h * in.head;
      const ET* pg = static_cast<const ET*>(grad.p) + int64_t(t) * grad.token + h * grad.head;
      float u[8] = {}, g[8] = {};
      load_pairs8<VEC>(px, e0, a.D, 0, a.layout, u, g);
      if (e0 < a.D) turned8<VEC>(pg, e0, a.D, a.rotary, a.layout, cs[buf], g);
      const float r = inverse_norm(u, a.D, a.norm.eps, lanes);
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
      const float c = group_sum(dot, lanes) / float(a.D);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = r * (y[j] - u[j] * c);
      if (e0 < a.D) put8<VEC>(static_cast<ET*>(out.p) + int64_t(t) * out.token + h * out.head, e0, a.D, y);
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

}  // namespace

int norm_parts(int T) { return T < kMostParts ? T : kMostParts; }

hipError_t launch_norm(const NormRopeArgs& a, int dtype, hipStream_t stream) {
  const dim3 grid(a.T), block(kRopeThreads);
  if (dtype == SV_BF16) {
    if (vec_of(a, 2, false))
      hipLaunchKernelGGL((norm_rope_kernel<true, uint16_t>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((norm_rope_kernel<false, uint16_t>), grid, block, 0, stream, a);
  } else {
    if (vec_of(a, 4, false))
      hipLaunchKernelGGL((norm_rope_kernel<true, float>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((norm_rope_kernel<false, float>), grid, block, 0, stream, a);
  }
  return hipGetLastError();
}

hipError_t launch_norm_backward(const NormRopeArgs& a, int dtype, hipStream_t stream) {
  const int parts = norm_parts(a.T);
  const dim3 grid(parts), block(kRopeThreads);
  if (parts > 0) {
    if (dtype == SV_BF16) {
      if (vec_of(a, 2, true))
        hipLaunchKernelGGL((norm_rope_backward_kernel<true, uint16_t>), grid, block, 0, stream, a);
      else
        hipLaunchKernelGGL((norm_rope_backward_kernel<false, uint16_t>), grid, block, 0, stream, a);
    } else {
      if (vec_of(a, 4, true))
        hipLaunchKernelGGL((norm_rope_backward_kernel<true, float>), grid, block, 0, stream, a);
      else
        hipLaunchKernelGGL((norm_rope_backward_kernel<false, float>), grid, block, 0, stream, a);
    }
  }
  if (a.dq_weight || a.dk_weight)
    hipLaunchKernelGGL(weight_gradient_kernel, dim3((2 * a.D + 15) / 16), dim3(kJoinThreads), 0, stream, a, parts);
  return hipGetLastError();
}

}  // namespace sv
