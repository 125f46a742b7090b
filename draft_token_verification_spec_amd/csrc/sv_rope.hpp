// Shared by the kernels that turn heads' rows: angles, rows of 8 channels a
// lane, and their way into a cache.
#pragma once

#include "sv_attn.hpp"

namespace sv {

constexpr int kRopeThreads = 256;
constexpr int kMaxPairs = SV_ATTN_MAX_HEAD_DIM / 2;

// Half turns of the angle position * f without its whole turns, in -1..1.
__device__ __forceinline__ double half_turns(double position, double f) {
  constexpr double kInv2Pi = 0.15915494309189535, kInv2PiLow = -9.839338337591243e-18;  // 1 / (2 pi) to 106 bits
  const double angle = position * f, low = fma(position, f, -angle);
  double turns = fma(angle, kInv2Pi, -rint(angle * kInv2Pi));
  turns += fma(angle, kInv2PiLow, low * kInv2Pi);
  return 2 * turns;
}

// mscale * (cos, sin) of the angle position * f.
__device__ __forceinline__ float2 turn_of(double position, double f, float mscale, float sign) {
  constexpr double kPi = 3.141592653589793;
  // what binary32 drops of the half turns is put back to first order
  const double halves = half_turns(position, f);
  const float near = float(halves), rest = float((halves - near) * kPi);
  float s, c;
  sincospif(near, &s, &c);
  return make_float2(fmaf(-rest, s, c) * mscale, fmaf(rest, c, s) * mscale * sign);
}

// The same of the row's angles, by the whole workgroup.
__device__ __forceinline__ void make_angles(float2* cs, const double* freq, int pairs, double position, float mscale,
                                            float sign) {
  for (int i = threadIdx.x; i < pairs; i += kRopeThreads) cs[i] = turn_of(position, freq[i], mscale, sign);
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

inline bool rows_vec(const void* p, int64_t token, int64_t head, int elem) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (token * elem) % 16 == 0 && (head * elem) % 16 == 0;
}

// Whole groups of 8 channels on either side of the turned channels' ends.
inline bool channels_vec(int D, int rotary, int layout) {
  return D % 8 == 0 && rotary % (layout == SV_ROPE_HALF ? 16 : 8) == 0;
}

}  // namespace sv
