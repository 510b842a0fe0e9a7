// w8a8_quantize.hip -- per-token quantizer: x (M, K) fp32 / fp16 / bf16 to
// int8 codes and one fp32 scale for each row.
//
//   s = max |x| / 127 (fp32, correctly rounded)
//   q = clamp(rint(x / s), -127, 127), the quotient taken exactly
//
// A group of waves owns a row: one pass takes the largest magnitude as the
// largest bit pattern without its sign (NaN > infinity > finite, so one
// integer maximum also finds rows that are not finite), a second forms the
// codes, the row held in registers between them where it fits.
//
// rint of the exact quotient at the cost of a multiply: f = x fl(1 / s) is
// within |x / s| 2^-22 of the quotient, so unless f is within |f| 2^-20 of a
// half both round alike.  For the few that are that near, with h the half,
// the sign of fma(-h, s, x) is the sign of x / s - h (a fused multiply-add rounds
// a nonzero value to a nonzero one), and 0 is a tie.  Rows whose scale is so
// small that 1 / s would overflow are lifted by 2^64 first, which is exact.
#include <type_traits>

#include "w8a8_device.h"

namespace qmm {

template <int XDT> struct Elem;
template <> struct Elem<XF16> { typedef _Float16 type; };
template <> struct Elem<XBF16> { typedef __bf16 type; };
template <> struct Elem<YF32> { typedef float type; };

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)v, d);
    v = o > v ? o : v;
  }
  return v;
}

// 8 elements of a row from element k on (zeros past K).
template <int XDT, bool VEC>
__device__ __forceinline__ void load8(const typename Elem<XDT>::type* row, int k, int K,
                                      float (&v)[8]) {
  typedef typename Elem<XDT>::type T;
  if (VEC && k + 8 <= K) {
    if constexpr (XDT == YF32) {
      const f32x4_t a = *reinterpret_cast<const f32x4_t*>(row + k);
      const f32x4_t b = *reinterpret_cast<const f32x4_t*>(row + k + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
    } else {
      typedef T T8 __attribute__((ext_vector_type(8)));
      const T8 a = *reinterpret_cast<const T8*>(row + k);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (float)a[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = k + j < K ? (float)row[k + j] : 0.0f;
  }
}

__device__ __forceinline__ float code_of(float x, float s, float r) {
  const float f = x * r;
  float q = __builtin_rintf(f);
  const float lo = __builtin_floorf(f);
  if (fabsf(f - lo - 0.5f) <= fabsf(f) * 0x1p-20f) {
    const float d = __builtin_fmaf(-(lo + 0.5f), s, x);
    const float even = 2.0f * __builtin_rintf(0.5f * lo);  // of lo and lo + 1, or a neighbour
    q = d > 0.0f ? lo + 1.0f : (d < 0.0f ? lo : (even == lo ? lo : lo + 1.0f));
  }
  return __builtin_amdgcn_fmed3f(q, -127.0f, 127.0f);
}

// WPR waves per row, HELD vectors of 8 elements per lane kept in registers
// (0: the row is read twice).
template <int XDT, int WPR, int HELD, bool VEC>
__global__ __launch_bounds__(256) void quantize_tokens_kernel(
    const typename Elem<XDT>::type* __restrict__ x, int64_t ldx, int8_t* __restrict__ xq,
    int64_t ldxq, float* __restrict__ sx, int M, int K) {
  constexpr int RPB = 4 / WPR;  // rows per workgroup
  __shared__ uint32_t part[4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = (int)blockIdx.x * RPB + wave / WPR;
  const bool live = m < M;
  const int t = (wave % WPR) * 64 + lane;
  constexpr int STEP = WPR * 64 * 8;
  const typename Elem<XDT>::type* row = x + (int64_t)(live ? m : 0) * ldx;

  float v[HELD > 0 ? HELD : 1][8];
  uint32_t top = 0;
  auto take = [&](const float (&e)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = __builtin_bit_cast(uint32_t, e[j]) & 0x7FFFFFFFu;
      top = b > top ? b : top;
    }
  };
  if constexpr (HELD > 0) {
#pragma unroll
    for (int i = 0; i < HELD; ++i) load8<XDT, VEC>(row, i * STEP + 8 * t, K, v[i]);
#pragma unroll
    for (int i = 0; i < HELD; ++i) take(v[i]);
  } else {
    for (int k = 8 * t; k < K; k += STEP) {
      load8<XDT, VEC>(row, k, K, v[0]);
      take(v[0]);
    }
  }
  top = wave_max_u32(top);
  if constexpr (WPR > 1) {
    if (lane == 0) part[wave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      const uint32_t o = part[(wave / WPR) * WPR + w];
      top = o > top ? o : top;
    }
  }
  if (!live) return;

  const bool bad = top >= 0x7F800000u;
  const float s = bad ? __builtin_nanf("") : __fdiv_rn(__builtin_bit_cast(float, top), 127.0f);
  if (t == 0) sx[m] = s;
  const bool none = bad || s == 0.0f;
  const float lift = s < 0x1p-100f ? 0x1p64f : 1.0f;
  const float ss = s * lift;
  const float r = __fdiv_rn(1.0f, none ? 1.0f : ss);
  const int K16 = (K + 15) & ~15;
  int8_t* qrow = xq + (int64_t)m * ldxq;
  auto put = [&](const float (&e)[8], int k) {
    if (k >= K16) return;
    uint32_t w[2] = {0u, 0u};
    if (!none) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        w[j / 4] |= ((uint32_t)(int)code_of(e[j] * lift, ss, r) & 0xFFu) << (8 * (j % 4));
    }
    *reinterpret_cast<u32x2_t*>(qrow + k) = u32x2_t{w[0], w[1]};
  };
  if constexpr (HELD > 0) {
#pragma unroll
    for (int i = 0; i < HELD; ++i) put(v[i], i * STEP + 8 * t);
  } else {
    for (int k = 8 * t; k < K16; k += STEP) {
      load8<XDT, VEC>(row, k, K, v[0]);
      put(v[0], k);
    }
  }
}

// ---------------------------------------------------------------- host side
template <int XDT, int WPR, int HELD>
static hipError_t launch_q(const void* x, int64_t ldx, int8_t* xq, int64_t ldxq, float* sx, int M,
                           int K, hipStream_t s) {
  typedef typename Elem<XDT>::type T;
  const bool vec = (reinterpret_cast<uintptr_t>(x) % 16) == 0 && (ldx * sizeof(T)) % 16 == 0;
  const dim3 grid((unsigned)(((int64_t)M * WPR + 3) / 4)), block(256);
  return vec ? launch_kernel(quantize_tokens_kernel<XDT, WPR, HELD, true>, grid, block, s,
                             static_cast<const T*>(x), ldx, xq, ldxq, sx, M, K)
             : launch_kernel(quantize_tokens_kernel<XDT, WPR, HELD, false>, grid, block, s,
                             static_cast<const T*>(x), ldx, xq, ldxq, sx, M, K);
}

template <int XDT>
static hipError_t launch_q_type(const void* x, int64_t ldx, int8_t* xq, int64_t ldxq, float* sx,
                                int M, int K, hipStream_t s) {
  // a wave per row up to 512 elements, else a workgroup, the row held in
  // registers up to 16384 elements
  if (K <= 512) return launch_q<XDT, 1, 1>(x, ldx, xq, ldxq, sx, M, K, s);
  if (K <= 2048) return launch_q<XDT, 4, 1>(x, ldx, xq, ldxq, sx, M, K, s);
  if (K <= 4096) return launch_q<XDT, 4, 2>(x, ldx, xq, ldxq, sx, M, K, s);
  if (K <= 8192) return launch_q<XDT, 4, 4>(x, ldx, xq, ldxq, sx, M, K, s);
  if (K <= 16384) return launch_q<XDT, 4, 8>(x, ldx, xq, ldxq, sx, M, K, s);
  return launch_q<XDT, 4, 0>(x, ldx, xq, ldxq, sx, M, K, s);
}

hipError_t launch_quantize_tokens(const void* x, int x_dtype, int64_t ldx, int8_t* xq,
                                  int64_t ldxq, float* sx, int M, int K, hipStream_t s) {
  if (x_dtype == YF32) return launch_q_type<YF32>(x, ldx, xq, ldxq, sx, M, K, s);
  if (x_dtype == XF16) return launch_q_type<XF16>(x, ldx, xq, ldxq, sx, M, K, s);
  return launch_q_type<XBF16>(x, ldx, xq, ldxq, sx, M, K, s);
}

}  // namespace qmm
