// Causal attention of packed new tokens over a paged cache.
//
// One workgroup per row and query head: a thread scores one token of a block
// of 256 at a time, the softmax runs online (running maximum and sum), and the
// weighted values are summed with a thread per channel.
#include "sv_attn.hpp"

namespace sv {

namespace {

constexpr int kAttnThreads = 256;

template <bool FP8>
__device__ __forceinline__ void cache8(const void* base, int64_t off, uint32_t biased, float (&x)[8]) {
  uint4 w;
  if (FP8)
    w = dequant8(*reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(base) + off), scale_of(biased));
  else
    w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + off);
  x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
  x[4] = bf16_lo(w.z), x[5] = bf16_hi(w.z), x[6] = bf16_lo(w.w), x[7] = bf16_hi(w.w);
}

template <bool FP8>
__global__ __launch_bounds__(kAttnThreads) void attention_kernel(AttnArgs a) {
  __shared__ float q[SV_ATTN_MAX_HEAD_DIM];
  __shared__ float p[kAttnThreads];
  __shared__ int pages[kAttnThreads];
  __shared__ float red[kAttnThreads / 64];
  const PagedView& c = a.cache;
  const int t = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, lane = tid & 63;
  const int b = find_sequence(a.query_start, a.B, t, lane);
  if (b < 0 || t >= a.query_start[b + 1]) return;
  const int64_t cap = int64_t(c.max_pages) << c.page_shift;
  const int held = int(max(int64_t(0), min(int64_t(a.kv_len[b]), cap)));
  const int place = int(uint32_t(a.kv_len[b]) - uint32_t(a.query_start[b + 1] - t));
  const int end = int(min(int64_t(place) + 1, int64_t(held)));
  const int begin = a.window > 0 ? max(0, int(max(int64_t(0), int64_t(place) + 1 - a.window))) : 0;
  const int kvh = h / (a.q_heads / c.heads);
  if (tid < c.D) q[tid] = load1(static_cast<const uint16_t*>(a.q.p) + t * a.q.token + h * a.q.head + tid) * (a.scale * kLog2e);
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int j0 = begin; j0 < end; j0 += kAttnThreads) {
    __syncthreads();
    const int j = j0 + tid;
    const int page = j < end ? page_of(c, b, j) : -1;
    const int slot = j & ((1 << c.page_shift) - 1);
    float s = -INFINITY;
    if (page >= 0) {
      s = 0.f;
      const int64_t off = page * c.k_page + slot * c.k_token + kvh * c.k_head;
      const uint32_t biased = FP8 ? c.k_scale[((int64_t(page) * c.heads + kvh) << c.page_shift) + slot] : 0u;
      for (int e = 0; e < c.D; e += 8) {
        float k8[8];
        cache8<FP8>(c.k, off + e, biased, k8);
#pragma unroll
        for (int i = 0; i < 8; ++i) s += q[e + i] * k8[i];
      }
    }
    pages[tid] = page;
    float top = s == s ? s : INFINITY;  // a NaN score must not be passed over by the maximum
    for (int i = 32; i >= 1; i >>= 1) top = fmaxf(top, __shfl_xor(top, i, 64));
    if (lane == 0) red[tid >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    if (top == -INFINITY) continue;
    const float m2 = fmaxf(m, top);
    const float w = s == -INFINITY ? 0.f : fast_exp2(s - m2);
    p[tid] = w;
    const float keep = m == -INFINITY ? 0.f : fast_exp2(m - m2);
    m = m2;
    __syncthreads();
    if (lane == 0) red[tid >> 6] = 0.f;
    float sum = wave_sum(w);
    if (lane == 0) red[tid >> 6] = sum;
    __syncthreads();
    l = l * keep + red[0] + red[1] + red[2] + red[3];
    o *= keep;
    if (tid < c.D) {
      for (int i = 0; i < kAttnThreads && j0 + i < end; ++i) {
        if (pages[i] < 0) continue;
        const int sl = (j0 + i) & ((1 << c.page_shift) - 1);
        const int64_t off = pages[i] * c.v_page + sl * c.v_token + kvh * c.v_head;
        const uint32_t biased = FP8 ? c.v_scale[((int64_t(pages[i]) * c.heads + kvh) << c.page_shift) + sl] : 0u;
        float v8[8];
        cache8<FP8>(c.v, off + (tid & ~7), biased, v8);
        float v = v8[0];
#pragma unroll
        for (int k = 1; k < 8; ++k) v = (tid & 7) == k ? v8[k] : v;
        o += p[i] * v;
      }
    }
  }
  if (tid < c.D) store1(static_cast<uint16_t*>(a.out.p) + t * a.out.token + h * a.out.head + tid, l == 0.f ? 0.f : o / l);
  if (a.lse && tid == 0)
    a.lse[int64_t(t) * a.q_heads + h] = l == 0.f ? -INFINITY : (m + fast_log2(l)) * kLn2;
}

}  // namespace

hipError_t launch_attention(const AttnArgs& a, int cache_dtype, hipStream_t stream) {
  const dim3 grid(a.T, a.q_heads), block(kAttnThreads);
  if (cache_dtype == SV_E4M3)
    hipLaunchKernelGGL(attention_kernel<true>, grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL(attention_kernel<false>, grid, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace sv
