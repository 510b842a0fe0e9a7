// mx4_device.h -- device helpers of the microscaled 4-bit kernels (gfx950).
#pragma once
#include <type_traits>

#include "mx4_internal.h"
#include "w8a8_device.h"

namespace qmm {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// 2^(e - 127) of a scale byte: 0 is the subnormal 2^-127, 255 NaN.
__device__ __forceinline__ float scale_f32(uint32_t e) {
  const uint32_t b = e << 23;
  return __builtin_bit_cast(float, e == 0 ? 0x00400000u : e == 255 ? 0x7FC00000u : b);
}

// 8 codes times their scale as bf16, pairs in order: exact wherever bf16 has
// the value (code times power of two: all but the ends of its range).
__device__ __forceinline__ u32x4_t bf16_of_codes(uint32_t c, float scale) {
  u32x4_t o;
  o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0));
  o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1));
  o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2));
  o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3));
  return o;
}

// 8 values to 8 codes with a block's scale byte (255: codes 0): the hardware
// divides by the power of two, rounds to nearest even and holds to +-6.
__device__ __forceinline__ uint32_t codes_of8(const float (&v)[8], uint32_t e) {
  const float s = scale_f32(e == 255 ? 127 : e);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
  return e == 255 ? 0u : c;
}

// The scale byte of a block from the bit pattern of its largest magnitude.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  const uint32_t e = top >> 23;
  return e == 255 ? 255u : (e < 2 ? 0u : e - 2);
}

// Values k .. k + 7 of a row of K (zeros from K on).  VEC: on 16 bytes, K a multiple of 8.  Else they are loaded at once where
// they lie, global memory takes any alignment; the last ones of a row with those before them, which settle8 shifts out when
// all of a wave's loads are under way (value by value, 333 x 1001 fp32 to packed codes took 6.3 us, so 4.7).
template <int XDT, bool VEC>
__device__ __forceinline__ Raw8<XDT> take8(const typename Elem<XDT>::type* row, int k, int K) {
  Raw8<XDT> r = {};
  const int n = K - k;
  if constexpr (VEC) {
    if (n > 0) {
      const u32x4_t* v = reinterpret_cast<const u32x4_t*>(row + k);
      r.w[0] = v[0];
      if constexpr (XDT == YF32) r.w[1] = v[1];
    }
  } else if (n > 0 && K >= 8) {
    typedef u32x4_t words_t __attribute__((aligned(4)));
    typedef u32x4_t halves_t __attribute__((aligned(2)));
    const int back = n >= 8 ? 0 : 8 - n;
    const auto* v = reinterpret_cast<const typename std::conditional<XDT == YF32, words_t, halves_t>::type*>(row + k - back);
    r.w[0] = v[0];
    if constexpr (XDT == YF32) r.w[1] = v[1];
  } else if (n > 0) {
#pragma unroll
    for (int j = 0; j < 7; ++j) {
      if (j >= n) break;
      if constexpr (XDT == YF32) r.w[j / 4][j % 4] = __builtin_bit_cast(uint32_t, row[k + j]);
      else r.w[0][j / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, row[k + j]) << (16 * (j % 2));
    }
  }
  return r;
}

template <int XDT, bool VEC> __device__ __forceinline__ void settle8(Raw8<XDT>& r, int k, int K) {
  const int back = K < 8 || K - k <= 0 || K - k >= 8 ? 0 : 8 - (K - k);
  if (VEC || back == 0) return;
  constexpr int WORDS = XDT == YF32 ? 8 : 4;
  uint32_t w[WORDS];
#pragma unroll
  for (int j = 0; j < WORDS; ++j) w[j] = r.w[j / 4][j % 4];
  const int words = XDT == YF32 ? back : back / 2;
#pragma unroll
  for (int s = WORDS / 2; s > 0; s /= 2)
#pragma unroll
    for (int j = 0; j < WORDS; ++j) w[j] = (words & s) == 0 ? w[j] : j + s < WORDS ? w[j + s] : 0;
  if constexpr (XDT != YF32)
#pragma unroll
    for (int j = 0; j < WORDS; ++j) w[j] = (back & 1) == 0 ? w[j] : (w[j] >> 16) | (j + 1 < WORDS ? w[j + 1] << 16 : 0);
#pragma unroll
  for (int j = 0; j < WORDS; ++j) r.w[j / 4][j % 4] = w[j];
}

}  // namespace qmm
