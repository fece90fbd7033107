// Device helpers shared by the operators around a caller's paged KV cache:
// rows of eight elements, the 8-bit codes, positions to places.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace photon {

__device__ __forceinline__ uint32_t div_fast(uint32_t n, const FastDiv& f) {
  return (__umulhi(n, f.mul) + n) >> f.shift;
}

// Storage of a page element by kind (PHOTON_KV_*).
struct e4m3 {
  __nv_fp8_storage_t x;
};
template <typename C> struct KvKind;
template <> struct KvKind<float> { static constexpr bool narrow = false; };
template <> struct KvKind<bf16> { static constexpr bool narrow = false; };
template <> struct KvKind<e4m3> {
  static constexpr bool narrow = true;
  static constexpr float top = 448.f;
};
template <> struct KvKind<int8_t> {
  static constexpr bool narrow = true;
  static constexpr float top = 127.f;
};

__device__ __forceinline__ void unpack_bf16(float* v, uint32_t w) {
  v[0] = __uint_as_float(w << 16);
  v[1] = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void unpack4(float* v, uint32_t w, e4m3) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2 h(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3));
    const float2 f = __half22float2(h);
    v[2 * i] = f.x, v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void unpack4(float* v, uint32_t w, int8_t) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (float)(int8_t)(w >> (8 * i));
}
// Eight consecutive elements from fp32.  VEC: the address is aligned to 16
// bytes (8 for 8-bit elements).
template <bool VEC>
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  if constexpr (VEC) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = v[i];
  }
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool VEC>
__device__ __forceinline__ void store8(bf16* p, const float (&v)[8]) {
  if constexpr (VEC) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                              pack_bf16(v[6], v[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = __float2bfloat16_rn(v[i]);
  }
}
// Values already multiplied by top / amax: rounded to nearest, ties to even.
template <bool VEC>
__device__ __forceinline__ void store8(e4m3* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i], v[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}
// v rounded to a whole number (|v| below 2^22) in the low bits of the sum: the
// conversion instruction runs at a quarter of an addition's rate.
__device__ __forceinline__ uint32_t whole(float v) { return __float_as_uint(__fadd_rn(v, 12582912.f)); }
template <bool VEC>
__device__ __forceinline__ void store8(int8_t* p, const float (&v)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = __byte_perm(__byte_perm(whole(v[4 * i]), whole(v[4 * i + 1]), 0x0040),
                       __byte_perm(whole(v[4 * i + 2]), whole(v[4 * i + 3]), 0x0040), 0x5410);
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(bf16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store1(e4m3* p, float v) { p->x = __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3); }
__device__ __forceinline__ void store1(int8_t* p, float v) { *p = (int8_t)whole(v); }

// Page and row of position `pos` of a sequence; false where there is none
// (reported, so that nothing is read or written for it).
__device__ __forceinline__ bool page_of(const int* table, int width, const KvPoolArgs& p, int pos, int* page, int* row,
                                        int* err) {
  const uint32_t n = div_fast((uint32_t)pos, p.div);
  if (n >= (uint32_t)width) return report_error(err, DEV_BAD_PLACE), false;
  const int id = table[n];
  if ((uint32_t)id >= (uint32_t)p.pages) return report_error(err, DEV_BAD_PLACE), false;
  *page = id;
  *row = pos - (int)n * p.rows;
  return true;
}

}  // namespace photon
