// w8a8_device.h -- device helpers of the int8 x int8 kernels (gfx950).
#pragma once
#include "qmm_device.h"
#include "w8a8_internal.h"

namespace qmm {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

// e^v for fp32, within about two units in the last place over the whole
// range: v log2(e) as a rounded product and its remainder (one fused multiply-add,
// plus the part of log2(e) that fp32 drops), 2^p (1 + r ln 2) from the
// hardware's 2^p.  The bare 2^(v log2 e) loses |v| 2^-24 of the result.
// Arguments are clamped to where the result is 0 or infinite anyway, so that
// the remainder of an infinity is no NaN; a NaN stays one.
__device__ __forceinline__ float exp_f32(float v) {
  v = v > 200.0f ? 200.0f : v;
  v = v < -200.0f ? -200.0f : v;
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
// 1 - p is formed as e^-t / (1 + e^-t), which keeps its leading digits; v p
// is taken as 0 where p is, so that act(-inf) is 0 and not -inf * 0.
__device__ __forceinline__ float act_parts(int act, float v, float* dact) {
  if (act == ACT_GELU) {
    const float p = 0.5f * erfcf(v * -0.707106781f);
    const float d = exp_f32(-0.5f * v * v) * 0.398942280f;
    const float vd = d == 0.0f ? 0.0f : v * d;
    *dact = p + vd;
    return p == 0.0f ? 0.0f : v * p;
  }
  const float c2 = 1.59576912f;  // 2 sqrt(2 / pi)
  const float t = act == ACT_SILU ? v : c2 * __builtin_fmaf(0.044715f * v * v, v, v);
  const float dt = act == ACT_SILU ? 1.0f : c2 * __builtin_fmaf(0.134145f * v, v, 1.0f);
  // with e = e^-|t|: p = 1 / (1 + e) or e / (1 + e), 1 - p the other
  const float e = exp_f32(-fabsf(t));
  const float r = 1.0f / (1.0f + e);
  const float lo = e * r;
  const float p = t >= 0.0f ? r : (t < 0.0f ? lo : t);  // NaN stays
  const float pq = r * lo;
  const float vd = pq == 0.0f ? 0.0f : v * pq * dt;
  *dact = p + vd;
  return p == 0.0f ? 0.0f : v * p;
}

// The 16-bit types of gradients, by their code.
template <int DT> struct Half16;
template <> struct Half16<XF16> { typedef _Float16 type; };
template <> struct Half16<XBF16> { typedef __bf16 type; };

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

}  // namespace qmm
