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
// How a code is rounded from the exact quotient: w8a8_device.h, code_of.
#include <type_traits>

#include "w8a8_device.h"

namespace qmm {

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
  typedef typename Elem<XDT>::type T;
  const buf_t row = make_buf(x + (int64_t)(live ? m : 0) * ldx, (uint32_t)(K * sizeof(T)));

  Raw8<XDT> v[HELD > 0 ? HELD : 1];
  uint32_t top = 0;
  if constexpr (HELD > 0) {
#pragma unroll
    for (int i = 0; i < HELD; ++i) v[i] = load8<XDT, VEC>(row, i * STEP + 8 * t);
#pragma unroll
    for (int i = 0; i < HELD; ++i) top = top8<XDT>(v[i], top);
  } else {
    for (int k = 8 * t; k < K; k += STEP) {
      v[0] = load8<XDT, VEC>(row, k);
      top = top8<XDT>(v[0], top);
    }
  }
  top = wave_max_u32(top_f32<XDT>(top));
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

  const RowScale c = row_scale(top);
  if (t == 0) sx[m] = c.s;
  const int K16 = (K + 15) & ~15;
  int8_t* qrow = xq + (int64_t)m * ldxq;
  auto put = [&](const Raw8<XDT>& e, int k) {
    if (k >= K16) return;
    *reinterpret_cast<u32x2_t*>(qrow + k) = codes8<XDT>(e, c);
  };
  if constexpr (HELD > 0) {
#pragma unroll
    for (int i = 0; i < HELD; ++i) put(v[i], i * STEP + 8 * t);
  } else {
    for (int k = 8 * t; k < K16; k += STEP) {
      v[0] = load8<XDT, VEC>(row, k);
      put(v[0], k);
    }
  }
}

// ---------------------------------------------------------------- host side
template <int XDT, int WPR, int HELD>
static hipError_t launch_q(const void* x, int64_t ldx, int8_t* xq, int64_t ldxq, float* sx, int M,
                           int K, hipStream_t s) {
  typedef typename Elem<XDT>::type T;
  const bool vec = vec8_ok(x, ldx, K, (int)sizeof(T));
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
  // registers up to 16384 elements (4096 x 4096 bf16: 4 waves to a row 13.9 us,
  // 2 waves 15.3, 1 wave 17.5; 4096 x 11008 28.1 us, 4.8 TB/s)
  if (K <= 512) return launch_q<XDT, 1, 1>(x, ldx, xq, ldxq, sx, M, K, s);
  if (K <= 2048) return launch_q<XDT, 4, 1>(x, ldx, xq, ldxq, sx, M, K, s);
  if (K <= 4096) return launch_q<XDT, 4, 2>(x, ldx, xq, ldxq, sx, M, K, s);
  if (K <= 8192) return launch_q<XDT, 4, 4>(x, ldx, xq, ldxq, sx, M, K, s);
  if (K <= 16384) return launch_q<XDT, 4, 8>(x, ldx, xq, ldxq, sx, M, K, s);
  return launch_q<XDT, 4, 0>(x, ldx, xq, ldxq, sx, M, K, s);
}

hipError_t launch_quantize_tokens(const void* x, int x_dtype, int64_t ldx, int8_t* xq,
                                  int64_t ldxq, float* sx, int M, int K, hipStream_t s) {
  hipError_t e = hipSuccess;
  for (int64_t m = 0; m < M && e == hipSuccess; m += kMaxLaunchRows) {
    const int rows = (int)(M - m < kMaxLaunchRows ? M - m : kMaxLaunchRows);
    const void* xm = static_cast<const char*>(x) + m * ldx * (x_dtype == YF32 ? 4 : 2);
    int8_t* qm = xq + m * ldxq;
    if (x_dtype == YF32) e = launch_q_type<YF32>(xm, ldx, qm, ldxq, sx + m, rows, K, s);
    else if (x_dtype == XF16) e = launch_q_type<XF16>(xm, ldx, qm, ldxq, sx + m, rows, K, s);
    else e = launch_q_type<XBF16>(xm, ldx, qm, ldxq, sx + m, rows, K, s);
  }
  return e;
}

}  // namespace qmm
