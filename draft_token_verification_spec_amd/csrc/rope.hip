// Rotary positions on their own, and with the append of new keys and values
// to a paged cache.
//
// Pair i of a head's first `rotary` channels is turned by the angle
// position * freq[i].  The angle is formed in binary64, with the product's
// rounding error carried along, as a number of turns (a position of 10^6 times
// a frequency of 1 leaves binary32 no fraction); its whole turns are dropped
// there, and cos and sin taken in binary32 of the remaining half turn at most,
// with what its rounding drops put back (an error near their own rounding's).
//
// One workgroup per row (new token): its rotary / 2 cos / sin pairs go to LDS
// once and serve every head.  A group of 8, 16 or 32 lanes takes a head, a
// lane 8 consecutive channels; it reads its pair's other channels itself (the
// line its neighbour just read), so that every lane makes one 16-byte store
// and a head's largest magnitude is a reduction over its group.
//
// Bound by HBM for many rows: 16381 rows of 32 heads of 128 binary32 channels,
// 537 MB read and written in 96.3 us (5.6 TB/s; a plain copy reaches 5.1); an
// append of 11311 rows of 32 + 8 + 8 heads of 128 to an 8-bit cache, 256 MB in
// 57.8 us (4.4 TB/s: 24-byte pieces of the cache and its scales besides).  By
// latency for few: 64 rows 3.4 us, an append of 1280 rows 9.4 us.  A workgroup
// per row rather than several rows keeps the angles' binary64 work (one pair a
// thread) off the heads' path; asking for a lane's later heads ahead cost more
// registers than it hid (an append took half as long again).
#include "sv_attn.hpp"

namespace sv {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxPairs = SV_ATTN_MAX_HEAD_DIM / 2;

// mscale * (cos, sin) of the row's angles, by the whole workgroup.
__device__ __forceinline__ void make_angles(float2* cs, const double* freq, int pairs, double position, float mscale,
                                            float sign) {
  constexpr double kInv2Pi = 0.15915494309189535, kInv2PiLow = -9.839338337591243e-18;  // 1 / (2 pi) to 106 bits
  constexpr double kPi = 3.141592653589793;
  for (int i = threadIdx.x; i < pairs; i += kRopeThreads) {
    const double f = freq[i], angle = position * f, low = fma(position, f, -angle);
    double turns = fma(angle, kInv2Pi, -rint(angle * kInv2Pi));
    turns += fma(angle, kInv2PiLow, low * kInv2Pi);
    // what binary32 drops of the half turns is put back to first order
    const double halves = 2 * turns;
    const float near = float(halves), rest = float((halves - near) * kPi);
    float s, c;
    sincospif(near, &s, &c);
    cs[i] = make_float2(fmaf(-rest, s, c) * mscale, fmaf(rest, c, s) * mscale * sign);
  }
}

// Channels e0 .. e0 + 7 of one head's row x, turned.  VEC: x is 16-byte
// aligned, D a multiple of 8, and the turned channels and pairs come in whole
// groups of 8.
template <bool VEC, typename ET>
__device__ __forceinline__ void turned8(const ET* x, int e0, int D, int rotary, int layout, const float2* cs,
                                        float (&y)[8]) {
  const int half = rotary >> 1;
  if (VEC) {
    load8(x + e0, y);
    if (e0 >= rotary) return;
    if (layout == SV_ROPE_HALF) {
      float z[8];
      const bool first = e0 < half;
      const int i0 = first ? e0 : e0 - half;
      load8(x + (first ? e0 + half : i0), z);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 w = cs[i0 + j];
        y[j] = first ? y[j] * w.x - z[j] * w.y : z[j] * w.y + y[j] * w.x;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float2 w = cs[(e0 + j) >> 1];
        const float a = y[j], c = y[j + 1];
        y[j] = a * w.x - c * w.y;
        y[j + 1] = a * w.y + c * w.x;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = e0 + j;
      y[j] = 0.f;
      if (e >= D) continue;
      y[j] = load1(x + e);
      if (e >= rotary) continue;
      const bool first = layout == SV_ROPE_HALF ? e < half : (e & 1) == 0;
      const int other = layout == SV_ROPE_HALF ? (first ? e + half : e - half) : e ^ 1;
      const float2 w = cs[layout == SV_ROPE_HALF ? (first ? e : e - half) : e >> 1];
      const float z = load1(x + other);
      y[j] = first ? y[j] * w.x - z * w.y : z * w.y + y[j] * w.x;
    }
  }
}

template <bool VEC, typename ET>
__device__ __forceinline__ void put8(ET* out, int e0, int D, const float (&y)[8]) {
  if (VEC) {
    store8(out + e0, y);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e0 + j < D) store1(out + e0 + j, y[j]);
  }
}

// log2 of the lanes that take a head.
__host__ __device__ inline int head_lanes_log2(int D) { return D <= 64 ? 3 : D <= 128 ? 4 : 5; }

template <bool VEC, typename ET>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a) {
  __shared__ float2 cs[kMaxPairs];
  const int t = blockIdx.x;
  make_angles(cs, a.freq, a.rotary >> 1, double(a.positions[t]), a.mscale, a.backward ? -1.f : 1.f);
  __syncthreads();
  const int lg = head_lanes_log2(a.D);
  const int e0 = (threadIdx.x & ((1 << lg) - 1)) * 8;
  if (e0 >= a.D) return;
  const ET* x = static_cast<const ET*>(a.x.p) + int64_t(t) * a.x.token;
  ET* out = static_cast<ET*>(a.out.p) + int64_t(t) * a.out.token;
  for (int h = threadIdx.x >> lg; h < a.heads; h += kRopeThreads >> lg) {
    float y[8];
    turned8<VEC>(x + h * a.x.head, e0, a.D, a.rotary, a.layout, cs, y);
    put8<VEC>(out + h * a.out.head, e0, a.D, y);
  }
}

// Least e >= -117 with amax <= 448 * 2^e: 448 = 0.875 * 2^9 (-9 for 0).  The
// type's smallest step, 2^-9, times 2^-117 is still a normal bf16 value.
__device__ __forceinline__ int scale_exponent(float amax) {
  if (amax == 0.f) return -9;
  int e;
  const float m = frexpf(amax, &e);
  return max(m > 0.875f ? e - 8 : e - 9, -117);
}

// 8 elements / 2^e as packed e4m3, nearest even; not finite: NaN.
__device__ __forceinline__ uint2 quant8(const float (&y)[8], int e) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float z[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      z[j] = ldexpf(y[4 * i + j], -e);
      z[j] = fabsf(z[j]) < INFINITY ? z[j] : NAN;
    }
    int p = __builtin_amdgcn_cvt_pk_fp8_f32(z[0], z[1], 0, false);
    p = __builtin_amdgcn_cvt_pk_fp8_f32(z[2], z[3], p, true);
    w[i] = uint32_t(p);
  }
  return make_uint2(w[0], w[1]);
}

// One head's 8 channels per lane into the cache; `lanes` is the group's size.
template <bool FP8>
__device__ __forceinline__ void put_cache(const PagedView& c, void* base, int64_t off, uint8_t* scale, int64_t scale_at,
                                          int e0, bool live, const float (&y)[8], int lanes) {
  if (FP8) {
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float m = fabsf(y[j]);
      top = fmaxf(top, live && m < INFINITY ? m : 0.f);
    }
    for (int o = lanes >> 1; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    const int e = scale_exponent(top);
    if (!live) return;
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + off + e0) = quant8(y, e);
    if (e0 == 0) scale[scale_at] = uint8_t(e + 127);
  } else if (live) {
    store8(static_cast<uint16_t*>(base) + off + e0, y);
  }
}

template <bool VEC, bool FP8, typename ET>
__global__ __launch_bounds__(kRopeThreads) void append_kernel(AppendArgs a) {
  __shared__ float2 cs[kMaxPairs];
  const int t = blockIdx.x;
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
  const int page = page_of(a.cache, b, place);
  const double position = a.positions ? double(a.positions[t]) : double(place);
  make_angles(cs, a.freq, a.rotary >> 1, position, a.mscale, 1.f);
  __syncthreads();

  const int D = a.cache.D, heads = a.cache.heads;
  const int lg = head_lanes_log2(D), lanes = 1 << lg;
  const int e0 = (threadIdx.x & (lanes - 1)) * 8;
  const bool live = e0 < D;
  const int slot = place & ((1 << a.cache.page_shift) - 1);
  const int total = a.q_heads + (page >= 0 ? 2 * heads : 0);
  for (int g = threadIdx.x >> lg; g < total; g += kRopeThreads >> lg) {
    float y[8] = {};
    if (g < a.q_heads) {
      if (!live) continue;
      turned8<VEC>(static_cast<const ET*>(a.q.p) + int64_t(t) * a.q.token + g * a.q.head, e0, D, a.rotary, a.layout, cs,
                   y);
      put8<VEC>(static_cast<ET*>(a.q_out.p) + int64_t(t) * a.q_out.token + g * a.q_out.head, e0, D, y);
    } else if (g < a.q_heads + heads) {
      const int h = g - a.q_heads;
      if (live)
        turned8<VEC>(static_cast<const ET*>(a.k.p) + int64_t(t) * a.k.token + h * a.k.head, e0, D, a.rotary, a.layout,
                     cs, y);
      put_cache<FP8>(a.cache, a.cache.k, page * a.cache.k_page + slot * a.cache.k_token + h * a.cache.k_head,
                     a.cache.k_scale, ((int64_t(page) * heads + h) << a.cache.page_shift) + slot, e0, live, y, lanes);
    } else {
      const int h = g - a.q_heads - heads;
      if (live)
        turned8<VEC>(static_cast<const ET*>(a.v.p) + int64_t(t) * a.v.token + h * a.v.head, e0, D, 0, a.layout, cs, y);
      put_cache<FP8>(a.cache, a.cache.v, page * a.cache.v_page + slot * a.cache.v_token + h * a.cache.v_head,
                     a.cache.v_scale, ((int64_t(page) * heads + h) << a.cache.page_shift) + slot, e0, live, y, lanes);
    }
  }
}

bool rows_vec(const void* p, int64_t token, int64_t head, int elem) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (token * elem) % 16 == 0 && (head * elem) % 16 == 0;
}

// Whole groups of 8 channels on either side of the turned channels' ends.
bool channels_vec(int D, int rotary, int layout) {
  return D % 8 == 0 && rotary % (layout == SV_ROPE_HALF ? 16 : 8) == 0;
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, int dtype, hipStream_t stream) {
  const int elem = dtype == SV_BF16 ? 2 : 4;
  const bool vec = channels_vec(a.D, a.rotary, a.layout) && rows_vec(a.x.p, a.x.token, a.x.head, elem) &&
                   rows_vec(a.out.p, a.out.token, a.out.head, elem);
  const dim3 grid(a.T), block(kRopeThreads);
  if (dtype == SV_BF16) {
    if (vec)
      hipLaunchKernelGGL((rope_kernel<true, uint16_t>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((rope_kernel<false, uint16_t>), grid, block, 0, stream, a);
  } else {
    if (vec)
      hipLaunchKernelGGL((rope_kernel<true, float>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((rope_kernel<false, float>), grid, block, 0, stream, a);
  }
  return hipGetLastError();
}

template <bool VEC, bool FP8>
static void append_of(const AppendArgs& a, int dtype, hipStream_t stream) {
  const dim3 grid(a.T), block(kRopeThreads);
  if (dtype == SV_BF16)
    hipLaunchKernelGGL((append_kernel<VEC, FP8, uint16_t>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((append_kernel<VEC, FP8, float>), grid, block, 0, stream, a);
}

hipError_t launch_append(const AppendArgs& a, int dtype, int cache_dtype, hipStream_t stream) {
  const int elem = dtype == SV_BF16 ? 2 : 4;
  bool vec = channels_vec(a.cache.D, a.rotary, a.layout) && rows_vec(a.k.p, a.k.token, a.k.head, elem) &&
             rows_vec(a.v.p, a.v.token, a.v.head, elem);
  if (a.q_heads > 0)
    vec = vec && rows_vec(a.q.p, a.q.token, a.q.head, elem) && rows_vec(a.q_out.p, a.q_out.token, a.q_out.head, elem);
  if (cache_dtype == SV_E4M3)
    vec ? append_of<true, true>(a, dtype, stream) : append_of<false, true>(a, dtype, stream);
  else
    vec ? append_of<true, false>(a, dtype, stream) : append_of<false, false>(a, dtype, stream);
  return hipGetLastError();
}

}  // namespace sv
