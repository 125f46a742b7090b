// Shared by the rotary, cache and attention kernels: element access, packed
// sequences and page lookups.
#pragma once

#include <math.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "../../include/specverify_attn.h"
#include "sv_device.hpp"

namespace sv {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// A cache and its page table as the kernels take them.
struct PagedView {
  const int32_t* table;
  int64_t table_stride;
  int max_pages, num_pages, heads, D;
  int page_shift;  // log2(page size)
  void* k;
  void* v;
  int64_t k_page, k_token, k_head;  // strides, elements
  int64_t v_page, v_token, v_head;
  uint8_t* k_scale;
  uint8_t* v_scale;
};

// Two floats rounded to nearest even, as packed bf16.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const bf16x2 p = __builtin_convertvector(f32x2{lo, hi}, bf16x2);
  return __builtin_bit_cast(uint32_t, p);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 8 consecutive elements as floats: vector loads (16-byte aligned), or one by
// one the first n of them (the rest 0).
__device__ __forceinline__ void load8(const uint16_t* p, float (&x)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
  x[4] = bf16_lo(w.z), x[5] = bf16_hi(w.z), x[6] = bf16_lo(w.w), x[7] = bf16_hi(w.w);
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(uint16_t* p, float x) { *p = uint16_t(pack_bf16(x, 0.f)); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }

// The scale 2^e of a biased exponent byte (0 stands for 2^-127, a subnormal).
__device__ __forceinline__ float scale_of(uint32_t biased) {
  return __uint_as_float(biased ? biased << 23 : 1u << 22);
}

// 8 packed e4m3 elements times a power-of-two scale, as packed bf16: exact,
// since a value has 4 significant bits (bf16 has 8).
__device__ __forceinline__ uint4 dequant8(uint2 q, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q.x, scale, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q.x, scale, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q.y, scale, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q.y, scale, true);
  return make_uint4(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, c),
                    __builtin_bit_cast(uint32_t, d));
}

// The last sequence b of [0, B) with start[b] <= row, or -1: a 64-ary search
// by the whole wave (every lane returns it), one round trip for B <= 64, two
// for B <= 4096.  Any contents of start end it with a value in -1 .. B - 1.
__device__ __forceinline__ int find_sequence(const int32_t* start, int B, int row, int lane) {
  int lo = 0, hi = B;
  while (lo < hi) {
    const int step = (hi - lo + 63) >> 6;
    const int at = lo + lane * step;
    const bool in = at < hi;
    const int n = __popcll(__ballot(in && start[in ? at : lo] <= row));
    if (n == 0) break;
    const int base = lo;
    lo = base + (n - 1) * step + 1;
    hi = min(hi, base + n * step);
  }
  return lo - 1;
}

// The page that holds a place of sequence b, or -1: places outside the page
// table and pages outside the cache hold nothing.
__device__ __forceinline__ int page_of(const PagedView& c, int b, int place) {
  const int i = place >> c.page_shift;
  if (place < 0 || i >= c.max_pages) return -1;
  const int page = c.table[int64_t(b) * c.table_stride + i];
  return uint32_t(page) < uint32_t(c.num_pages) ? page : -1;
}

}  // namespace sv
