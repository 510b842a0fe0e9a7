// w8a8_device.h -- device helpers of the int8 x int8 kernels (gfx950).
#pragma once
#include <type_traits>

#include "qmm_device.h"
#include "w8a8_internal.h"

namespace qmm {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

// e^v, v <= 0, within about two units in the last place: v log2(e) as a rounded product and its remainder (one fused multiply-add,
// plus the part of log2(e) that fp32 drops), 2^p (1 + r ln 2) from the
// hardware's 2^p.  The bare 2^(v log2 e) loses |v| 2^-24 of the result.
// For v <= 0: below -200 the result is 0 anyway, and held there the remainder of
// an infinity is no NaN.  (A NaN gives 0 or 1: callers carry it otherwise.)
__device__ __forceinline__ float exp_f32(float v) {
  v = fmaxf(v, -200.0f);
  const float L = 1.44269504f, Llo = 1.925963033e-8f;  // log2(e) = L + Llo
  const float p = v * L;
  const float r = __builtin_fmaf(v, L, -p) + v * Llo;
  const float e = __builtin_amdgcn_exp2f(p);
  return __builtin_fmaf(e, r * 0.693147181f, e);
}

// act(v) = v p(v), and act'(v) = p + v p'.
//   silu: p = 1 / (1 + e^-v), p' = p (1 - p)
//   gelu: p = (1 + erf(v / sqrt 2)) / 2, p' = e^(-v^2 / 2) / sqrt(2 pi)
//   gelu_tanh: (1 + tanh z) / 2 = 1 / (1 + e^-2z), z = sqrt(2 / pi) (v + 0.044715 v^3),
//     p' = p (1 - p) 2 z'
// With e = e^-|t|, p and 1 - p are 1 / (1 + e) and e / (1 + e), either way round:
// both keep their leading digits.  v is held to +-1e30 where it meets a factor
// that may be 0, so that act(-inf) is 0 and no infinity times 0 appears; NaN comes
// back through p.
template <int ACT>
__device__ __forceinline__ float act_parts(float v, float* dact) {
  const float vlo = fmaxf(v, -1e30f), vc = fminf(vlo, 1e30f);
  if constexpr (ACT == ACT_GELU) {
    const float p = 0.5f * erfcf(v * -0.707106781f);
    const float d = exp_f32(-0.5f * vc * vc) * 0.398942280f;
    *dact = __builtin_fmaf(vc, d, p);
    return vlo * p;
  } else {
    const float c2 = 1.59576912f;  // 2 sqrt(2 / pi)
    const float t = ACT == ACT_SILU ? v : c2 * __builtin_fmaf(0.044715f * v * v, v, v);
    const float e = exp_f32(-fabsf(t));
    // 1 / (1 + e): the hardware's reciprocal and one Newton step
    const float d = 1.0f + e;
    const float r0 = __builtin_amdgcn_rcpf(d);
    const float r = __builtin_fmaf(__builtin_fmaf(-d, r0, 1.0f), r0, r0);
    const float lo = e * r;
    const float p = t >= 0.0f ? r : (t < 0.0f ? lo : t);  // NaN stays
    const float vq = vc * (r * lo);
    if constexpr (ACT == ACT_SILU) {
      *dact = p + vq;
    } else {
      const float dt = c2 * __builtin_fmaf(0.134145f * vc, vc, 1.0f);
      *dact = p + (r * lo == 0.0f ? 0.0f : vq * dt);
    }
    return vlo * p;
  }
}

// f with the activation as a constant (uniform across the launch).
template <class F> __device__ __forceinline__ void with_act(int act, F&& f) {
  if (act == ACT_SILU) f(std::integral_constant<int, ACT_SILU>{});
  else if (act == ACT_GELU) f(std::integral_constant<int, ACT_GELU>{});
  else f(std::integral_constant<int, ACT_GELU_TANH>{});
}

// The 16-bit types of gradients, by their code.
template <int DT> struct Half16;
template <> struct Half16<XF16> { typedef _Float16 type; };
template <> struct Half16<XBF16> { typedef __bf16 type; };

// ---- powers of two of fp16 operands -----------------------------------------
// Values that become fp16 operands are first multiplied by a power of two that their
// own block shares.  A block's level e is the exponent field of its largest magnitude
// (of an infinity 255, a NaN counts for nothing), rounded up to 7 mod 8, at least 31:
// the power 2^(141 - e) brings the largest value to [2^7, 2^15), where 21 binary digits
// below it are still normal numbers.  Steps of 8 because blocks of one row whose levels
// agree need not be touched again (w8a8_backward.hip).
__device__ __forceinline__ uint32_t level_of(float top) {
  const uint32_t e = (__builtin_bit_cast(uint32_t, top) >> 23) | 7u;
  return e < 31u ? 31u : e;
}
__device__ __forceinline__ float level_power(uint32_t e) {
  return __builtin_bit_cast(float, (268u - e) << 23);
}
__device__ __forceinline__ float level_inverse(uint32_t e) {
  return __builtin_bit_cast(float, (e - 14u) << 23);
}

// Largest of the values of 8 (16) consecutive lanes, in each of them.
template <int CTRL> __device__ __forceinline__ float dpp_max(float v) {
  const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false);
  return fmaxf(v, __builtin_bit_cast(float, o));
}
template <int LANES> __device__ __forceinline__ float lanes_max(float v) {
  static_assert(LANES == 8 || LANES == 16, "lanes of a DPP row");
  v = dpp_max<0xB1>(v);                     // quad_perm [1,0,3,2]
  v = dpp_max<0x4E>(v);                     // quad_perm [2,3,0,1]
  v = dpp_max<0x141>(v);                    // row_half_mirror
  if (LANES == 16) v = dpp_max<0x128>(v);   // row_ror:8
  return v;
}
// Largest over the wave's 4 rows of 16 lanes at each lane position, by two lane
// swaps (as rows4_sum).
__device__ __forceinline__ float rows4_max(float v) {
  float a0 = v, a1 = v;
  asm volatile("s_nop 1\n\tv_permlane16_swap_b32 %0, %1" : "+v"(a0), "+v"(a1));
  float c0 = fmaxf(a0, a1), c1 = c0;
  asm volatile("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(c0), "+v"(c1));
  return fmaxf(c0, c1);
}

// 4 consecutive values stored as the output type: one store where `vec`
// says that the address is aligned and all 4 exist, else one by one up to n.
template <class T>
__device__ __forceinline__ void store4(T* p, const float (&v)[4], int n, bool vec) {
  typedef T T4 __attribute__((ext_vector_type(4)));
  if (vec && n >= 4) {
    T4 o = {(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
    *reinterpret_cast<T4*>(p) = o;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) p[j] = (T)v[j];
  }
}

// True where 4-element stores (or loads) of elements of `size` bytes are
// aligned for every row of a matrix whose columns are taken in fours.
__device__ __forceinline__ bool vec4_ok(const void* p, int64_t ld, int size) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * size)) & (uintptr_t)(4 * size - 1)) == 0;
}

// The 16 bytes of a chunk that starts at contracted byte k, those from kb on
// cleared.
__device__ __forceinline__ u32x4_t clear_tail(u32x4_t v, int k, int kb) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int left = kb - (k + 4 * j);
    if (left <= 0) v[j] = 0;
    else if (left < 4) v[j] &= (1u << (8 * left)) - 1u;
  }
  return v;
}

// ---- quantizing rows ---------------------------------------------------------
template <int XDT> struct Elem;
template <> struct Elem<XF16> { typedef _Float16 type; };
template <> struct Elem<XBF16> { typedef __bf16 type; };
template <> struct Elem<YF32> { typedef float type; };

// Largest of the wave's 64 values, in every lane (DPP: butterfly inside each
// row of 16 lanes, then the rows' results broadcast into lane 63).
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#define QMM_DPP_MAX(ctrl, mask)                                                        \
  {                                                                                    \
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, mask, 0xF, false); \
    v = o > v ? o : v;                                                                 \
  }
  QMM_DPP_MAX(0xB1, 0xF)   // quad_perm [1,0,3,2]
  QMM_DPP_MAX(0x4E, 0xF)   // quad_perm [2,3,0,1]
  QMM_DPP_MAX(0x124, 0xF)  // row_ror:4
  QMM_DPP_MAX(0x128, 0xF)  // row_ror:8
  QMM_DPP_MAX(0x142, 0xA)  // row_bcast:15 into rows 1 and 3
  QMM_DPP_MAX(0x143, 0xC)  // row_bcast:31 into rows 2 and 3
#undef QMM_DPP_MAX
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// 8 consecutive elements as loaded: one 16-byte word of 16-bit elements, two
// of fp32 ones.
template <int XDT> struct Raw8 { u32x4_t w[XDT == YF32 ? 2 : 1]; };

// Elements k .. k + 7 of the row that buffer b ends with (zeros past its
// end): whole 16-byte loads, or one load per element where the row does not
// start on 16 bytes or end on them.
template <int XDT, bool VEC>
__device__ __forceinline__ Raw8<XDT> load8(buf_t b, int k) {
  Raw8<XDT> r;
  constexpr int SZ = XDT == YF32 ? 4 : 2;
  if constexpr (VEC) {
    r.w[0] = buf_load128(b, k * SZ);
    if constexpr (XDT == YF32) r.w[1] = buf_load128(b, k * SZ + 16);
  } else if constexpr (XDT == YF32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) r.w[j / 4][j % 4] = buf_load32(b, (k + j) * SZ);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      r.w[0][j] = buf_load16(b, (k + 2 * j) * SZ) | (buf_load16(b, (k + 2 * j + 1) * SZ) << 16);
  }
  return r;
}
// Whether whole 16-byte loads serve rows of K elements of `size` bytes.
__host__ __device__ inline bool vec8_ok(const void* x, int64_t ld, int K, int size) {
  return ((reinterpret_cast<uintptr_t>(x) | (uintptr_t)(ld * size) | (uintptr_t)((int64_t)K * size)) & 15) == 0;
}

template <int XDT>
__device__ __forceinline__ void floats8(const Raw8<XDT>& r, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (XDT == YF32) {
      const uint32_t e = r.w[j / 4][j % 4];
      v[j] = __builtin_bit_cast(float, e);
    } else if constexpr (XDT == XBF16) {
      const uint32_t e = r.w[0][j / 2];
      v[j] = __builtin_bit_cast(float, j % 2 ? e & 0xFFFF0000u : e << 16);
    } else {
      const uint32_t e = r.w[0][j / 2];
      const half2_t h = __builtin_bit_cast(half2_t, e);
      v[j] = (float)h[j % 2];
    }
  }
}

// Largest magnitude as bit patterns without the sign: they order as the
// values do, NaN above infinity above what is finite.  16-bit elements are
// compared in pairs, as they were loaded; top_f32 gives the fp32 pattern.
template <int XDT>
__device__ __forceinline__ uint32_t top8(const Raw8<XDT>& r, uint32_t top) {
  if constexpr (XDT == YF32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = r.w[j / 4][j % 4] & 0x7FFFFFFFu;
      top = b > top ? b : top;
    }
    return top;
  } else {
    typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
    u16x2_t t = __builtin_bit_cast(u16x2_t, top);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t b = r.w[0][j] & 0x7FFF7FFFu;
      t = __builtin_elementwise_max(t, __builtin_bit_cast(u16x2_t, b));
    }
    return __builtin_bit_cast(uint32_t, t);
  }
}
template <int XDT> __device__ __forceinline__ uint32_t top_f32(uint32_t top) {
  if constexpr (XDT == YF32) return top;
  const uint32_t lo = top & 0xFFFFu, hi = top >> 16, m = lo > hi ? lo : hi;
  if constexpr (XDT == XBF16) return m << 16;
  const float f = (float)__builtin_bit_cast(_Float16, (uint16_t)m);
  return __builtin_bit_cast(uint32_t, f);
}

// A row's scale from its largest magnitude, and what its codes are formed
// with: 1 / s, and for scales so small that this would overflow a factor
// 2^64 on both s and x first, which is exact.
struct RowScale {
  float s;     // as stored: NaN where the row is not finite
  float ss;    // s lift
  float r;     // 1 / ss
  float lift;  // 1 or 2^64
  bool none;   // every code is 0
};
__device__ __forceinline__ RowScale row_scale(uint32_t top) {
  RowScale c;
  const bool bad = top >= 0x7F800000u;
  c.s = bad ? __builtin_nanf("") : __fdiv_rn(__builtin_bit_cast(float, top), 127.0f);
  c.none = bad || c.s == 0.0f;
  c.lift = c.s < 0x1p-100f ? 0x1p64f : 1.0f;
  c.ss = c.s * c.lift;
  c.r = __fdiv_rn(1.0f, c.none ? 1.0f : c.ss);
  return c;
}

// rint of the exact quotient x / s, ties to even, clamped.  q = rint(x fl(1/s))
// is at most one off; d = x - q s is exact (a fused multiply-add, and what is
// left has no more bits than s), so 2 |d| against s decides: more than s moves
// q one further, s itself is a tie.
__device__ __forceinline__ float code_of(float x, float s, float r) {
  const float q = __builtin_rintf(x * r);
  const float d = 2.0f * __builtin_fmaf(-q, s, x);
  const float a = fabsf(d);
  const bool move = a > s || (a == s && ((int)q & 1));
  return __builtin_amdgcn_fmed3f(move ? q + __builtin_copysignf(1.0f, d) : q, -127.0f, 127.0f);
}

// 8 codes of a row, packed.  f = x fl(1 / s) is within |f| 2^-22 < 2^-15 of the
// quotient: unless one of the 8 lies within 2^-14 of a half, both round alike,
// and adding 1.5 2^23 leaves rint(f) in the sum's low bits, its low byte the
// code (in ordinary rows |f| < 127.5: nothing to clamp).  Else, and where the
// row is lifted, all 8 take code_of.
template <int XDT>
__device__ __forceinline__ u32x2_t codes8(const Raw8<XDT>& raw, const RowScale& c) {
  if (c.none) return u32x2_t{0u, 0u};
  float v[8];
  floats8<XDT>(raw, v);
  uint32_t b[8];
  float worst = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float f = v[j] * c.r;
    const float t = f + 12582912.0f;
    worst = fmaxf(worst, fabsf(f - (t - 12582912.0f)));
    b[j] = __builtin_bit_cast(uint32_t, t);
  }
  if (worst > 0.5f - 0x1p-14f || c.lift != 1.0f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = (uint32_t)(int)code_of(v[j] * c.lift, c.ss, c.r);
  }
  // low bytes of four words, by two byte permutes and a third
  auto pack = [](uint32_t p, uint32_t q, uint32_t r, uint32_t s) {
    const uint32_t lo = __builtin_amdgcn_perm(q, p, 0x0C0C0400u), hi = __builtin_amdgcn_perm(s, r, 0x04000C0Cu);
    return lo | hi;
  };
  return u32x2_t{pack(b[0], b[1], b[2], b[3]), pack(b[4], b[5], b[6], b[7])};
}

}  // namespace qmm
