// Numbers of the 8-bit cache: e4m3 codes and the scale of a row.
#pragma once

#include "attn_parts.hpp"

namespace fk {

// Two neighbouring codes of a word (its upper two if HI) as fp32, exact.
template <bool HI> __device__ __forceinline__ floatx2_t e4m3_pair(uint32_t w) {
  return __builtin_amdgcn_cvt_pk_f32_fp8((int)w, HI);
}

// One code.
__device__ __forceinline__ float e4m3_get(uint8_t c) { return __builtin_amdgcn_cvt_f32_fp8(c, 0); }

// Codes of four numbers of at most 448 in magnitude, or NaN; nearest, ties to even.
__device__ __forceinline__ uint32_t e4m3_codes(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return (uint32_t)w;
}

__device__ __forceinline__ bool is_finite(float x) { return fabsf(x) < INFINITY; }

// Exponent of the smallest power of two s >= 2^-126 with 448 s >= most (finite, >= 0).
// 448 = 1.75 * 2^8: adding 0.25 of a binade carries into the exponent where the
// fraction is above 1.75.
__device__ __forceinline__ int scale_exponent(float most) {
  const int e = (int)((__builtin_bit_cast(uint32_t, most) + 0x1FFFFFu) >> 23) - 127 - 8;
  return most == 0.f ? 0 : (e < -126 ? -126 : e);
}

__device__ __forceinline__ float pow2(int e) {          // -126 <= e <= 127
  return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23);
}

// What a code stands for, rounded by the caller: numbers past dt's largest become it.
template <int DT> __device__ __forceinline__ float clamp_to(float x) {
  constexpr float most = DT == FK_F16 ? 65504.f : (DT == FK_BF16 ? 0x1.FEp127f : 0x1.FFFFFEp127f);
  return x != x ? x : fminf(fmaxf(x, -most), most);
}

}  // namespace fk
