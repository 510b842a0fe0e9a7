// mx4_quantize.hip -- values to microscaled 4-bit codes and back, and the
// layout of weights that the products read.  All three are bound by memory.
#include "mx4_device.h"

namespace qmm {

// Largest over the 4 lanes of a quad, in each of them.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false);
  v = o > v ? o : v;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false);
  return o > v ? o : v;
}

// 4 lanes on a block, 8 values each: a wave reads 512 consecutive values and
// writes 256 consecutive bytes of codes.  `units` 8-value units a row.
template <int XDT, bool VEC>
__global__ __launch_bounds__(256) void mx4_quantize_kernel(
    const typename Elem<XDT>::type* __restrict__ x, int64_t ldx, uint8_t* __restrict__ codes,
    int64_t ldc, uint8_t* __restrict__ scales, int64_t lds, uint32_t total, int units, int K) {
  const uint32_t u = blockIdx.x * 256u + threadIdx.x;
  if (u >= total) return;  // whole quads: units are multiples of 4
  const uint32_t m = u / (uint32_t)units;
  const int i = (int)(u - m * (uint32_t)units);
  Raw8<XDT> raw = take8<XDT, VEC>(x + (int64_t)m * ldx, 8 * i, K);
  settle8<XDT, VEC>(raw, 8 * i, K);
  const uint32_t e = scale_byte(quad_max(top_f32<XDT>(top8<XDT>(raw, 0u))));
  float v[8];
  floats8<XDT>(raw, v);
  *reinterpret_cast<uint32_t*>(codes + (int64_t)m * ldc + 4 * i) = codes_of8(v, e);
  uint8_t* s = scales + (int64_t)m * lds;
  const int b = i / 4;
  if (i % 4 == 0) s[b] = (uint8_t)e;
  // padding of the row of scales, by the last block's other lanes
  if (b == units / 4 - 1 && i % 4 != 0) {
    const int at = b + i % 4;
    if (at < (units / 4 + 3) / 4 * 4 && at < lds) s[at] = 0;
  }
}

// Values to codes in the packed layout (as a weight (M, K)): a wave takes a chunk of 512
// values of 4 rows, 8 values a lane.  (Blocks of zeros past K have scale byte 0, which is as good
// as 127; rows past M are never stored by who reads them.)
template <int XDT, bool VEC>
__global__ __launch_bounds__(256) void mx4_quantize_packed_kernel(
    const typename Elem<XDT>::type* __restrict__ x, int64_t ldx, uint8_t* __restrict__ w, uint32_t total, int M, int K) {
  const int lane = threadIdx.x & 63;
  const uint32_t u = blockIdx.x * 4u + (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (u >= total) return;
  const uint32_t chunks = (uint32_t)mx4_chunks(K);
  const uint32_t at = u / 4;  // chunk of the matrix; rows 4 (u % 4) .. + 3 of its strip
  const uint32_t strip = at / chunks;
  const int c = (int)(at - strip * chunks);
  uint8_t* o = w + (int64_t)at * kChunkBytes;
  Raw8<XDT> raw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = 16 * (int)strip + 4 * (int)(u % 4) + i, k = 512 * c + 8 * lane;
    raw[i] = take8<XDT, VEC>(x + (int64_t)(m < M ? m : 0) * ldx, m < M ? k : K, K);
  }
  // lane: quarter lane % 4 of block lane / 4 = 4 q + j
  const int q = lane >> 4, j = (lane >> 2) & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * (int)(u % 4) + i;
    if (16 * (int)strip + r < M) settle8<XDT, VEC>(raw[i], 512 * c + 8 * lane, K);
    const uint32_t e = scale_byte(quad_max(top_f32<XDT>(top8<XDT>(raw[i], 0u))));
    float v[8];
    floats8<XDT>(raw[i], v);
    *reinterpret_cast<uint32_t*>(o + 1024 * j + 256 * q + 16 * r + 4 * (lane & 3)) = codes_of8(v, e);
    // the scales of 4 blocks meet in the first of their 16 lanes
    uint32_t d = e;
    d |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)e, 0x104, 0xF, 0xF, true) << 8;   // row_shl:4
    d |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)e, 0x108, 0xF, 0xF, true) << 16;  // row_shl:8
    d |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)e, 0x10C, 0xF, 0xF, true) << 24;  // row_shl:12
    if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(o + 4096 + 64 * q + 4 * r) = d;
  }
}

// 8 values per thread.
template <class Y, bool VEC>
__global__ __launch_bounds__(256) void mx4_dequantize_kernel(
    const uint8_t* __restrict__ codes, int64_t ldc, const uint8_t* __restrict__ scales, int64_t lds,
    Y* __restrict__ y, int64_t ldy, uint32_t total, int units, int K) {
  const uint32_t u = blockIdx.x * 256u + threadIdx.x;
  if (u >= total) return;
  const uint32_t m = u / (uint32_t)units;
  const int i = (int)(u - m * (uint32_t)units);
  const uint8_t* p = codes + (int64_t)m * ldc + 4 * i;
  uint32_t c;
  if constexpr (VEC) c = *reinterpret_cast<const uint32_t*>(p);
  else c = p[0] | (p[1] << 8) | (p[2] << 16) | ((uint32_t)p[3] << 24);
  const float s = scale_f32(scales[(int64_t)m * lds + i / 4]);
  float v[8];
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0);
  const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
  const f32x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2);
  const f32x2_t f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3);
  v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1];
  v[4] = d[0], v[5] = d[1], v[6] = f[0], v[7] = f[1];
  Y* o = y + (int64_t)m * ldy + 8 * i;
  const int n = K - 8 * i;
  if (n >= 8) {
    typedef Y Y8 __attribute__((ext_vector_type(8)));
    Y8 q;
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = (Y)v[j];
    if constexpr (VEC) *reinterpret_cast<Y8*>(o) = q;
    else __builtin_memcpy(o, &q, sizeof(q));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) o[j] = (Y)v[j];
  }
}

// A thread writes 16 bytes of a packed chunk: a block's codes, or 4 columns' 4 scales.
__global__ __launch_bounds__(256) void mx4_pack_kernel(const uint8_t* __restrict__ codes, int64_t ldc,
                                                       const uint8_t* __restrict__ scales, int64_t lds,
                                                       u32x4_t* __restrict__ w, int strips, int N,
                                                       int K, int first) {
  const int blocks = mx4_blocks(K), chunks = mx4_chunks(K);
  constexpr int PER = kChunkBytes / 16;  // 256 of codes, 16 of scales
  const int pieces = PER * chunks;
  const int64_t strip = (int64_t)first + blockIdx.x;  // of all matrices
  const int64_t matrix = strip / strips;
  const int n0 = (int)(strip - matrix * strips) * 16;
  for (int i = (int)blockIdx.y * 256 + (int)threadIdx.x; i < pieces; i += (int)gridDim.y * 256) {
    const int c = i / PER, p = i - PER * c;
    u32x4_t o = {0u, 0u, 0u, 0u};
    if (p < 256) {
      const int n = n0 + p % 16, b = 16 * c + 4 * (p / 16 % 4) + p / 64;
      if (n < N && b < blocks) {
        const uint8_t* src = codes + (matrix * N + n) * ldc + 16 * b;
        if ((reinterpret_cast<uintptr_t>(src) & 15) == 0) {
          o = *reinterpret_cast<const u32x4_t*>(src);
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j / 4] |= (uint32_t)src[j] << (8 * (j % 4));
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int l = 4 * (p - 256) + j / 4, n = n0 + l % 16, b = 16 * c + 4 * (l / 16) + j % 4;
        const uint32_t e = n < N && b < blocks ? scales[(matrix * N + n) * lds + b] : 127u;
        o[j / 4] |= e << (8 * (j % 4));
      }
    }
    w[strip * pieces + i] = o;
  }
}

// ---------------------------------------------------------------- host side
// f(first row, rows) for launches of at most 2^31 units.
template <class F> static hipError_t by_rows(int M, int units, F&& f) {
  const int64_t rows = (int64_t(1) << 31) / units;
  hipError_t e = hipSuccess;
  for (int64_t m = 0; m < M && e == hipSuccess; m += rows)
    e = f(m, (int)(M - m < rows ? M - m : rows));
  return e;
}
static dim3 groups_of(uint32_t total) { return dim3((unsigned)(((int64_t)total + 255) / 256)); }

template <int XDT>
static hipError_t quantize_t(const void* x, int64_t ldx, uint8_t* codes, int64_t ldc, uint8_t* scales,
                             int64_t lds, int M, int K, hipStream_t s) {
  typedef typename Elem<XDT>::type T;
  const int units = 4 * mx4_blocks(K);
  const bool vec = vec8_ok(x, ldx, K, sizeof(T)) && K % 8 == 0;
  return by_rows(M, units, [&](int64_t m, int rows) {
    const uint32_t total = (uint32_t)rows * (uint32_t)units;
    return launch_kernel(vec ? mx4_quantize_kernel<XDT, true> : mx4_quantize_kernel<XDT, false>,
                         groups_of(total), dim3(256), s, static_cast<const T*>(x) + m * ldx, ldx,
                         codes + m * ldc, ldc, scales + m * lds, lds, total, units, K);
  });
}

hipError_t launch_mx4_quantize(const void* x, int x_dtype, int64_t ldx, uint8_t* codes, int64_t ldc,
                               uint8_t* scales, int64_t lds, int M, int K, hipStream_t s) {
  switch (x_dtype) {
    case XF16: return quantize_t<XF16>(x, ldx, codes, ldc, scales, lds, M, K, s);
    case XBF16: return quantize_t<XBF16>(x, ldx, codes, ldc, scales, lds, M, K, s);
  }
  return quantize_t<YF32>(x, ldx, codes, ldc, scales, lds, M, K, s);
}

template <int XDT>
static hipError_t quantize_packed_t(const void* x, int64_t ldx, uint8_t* w, int M, int K, hipStream_t s) {
  typedef typename Elem<XDT>::type T;
  const bool vec = vec8_ok(x, ldx, K, sizeof(T)) && K % 8 == 0;
  // strips of one launch: at most 2^25 waves
  const int64_t strips = ((int64_t)M + 15) / 16, most = (int64_t(1) << 23) / mx4_chunks(K);
  hipError_t e = hipSuccess;
  for (int64_t f = 0; f < strips && e == hipSuccess; f += most) {
    const int64_t n = strips - f < most ? strips - f : most;
    const uint32_t total = (uint32_t)(4 * n * mx4_chunks(K));
    e = launch_kernel(vec ? mx4_quantize_packed_kernel<XDT, true> : mx4_quantize_packed_kernel<XDT, false>,
                      dim3((total + 3) / 4), dim3(256), s, static_cast<const T*>(x) + 16 * f * ldx, ldx,
                      w + f * mx4_strip_bytes(K), total, (int)(M - 16 * f < 16 * n ? M - 16 * f : 16 * n), K);
  }
  return e;
}

hipError_t launch_mx4_quantize_packed(const void* x, int x_dtype, int64_t ldx, uint8_t* w, int M, int K,
                                      hipStream_t s) {
  switch (x_dtype) {
    case XF16: return quantize_packed_t<XF16>(x, ldx, w, M, K, s);
    case XBF16: return quantize_packed_t<XBF16>(x, ldx, w, M, K, s);
  }
  return quantize_packed_t<YF32>(x, ldx, w, M, K, s);
}

template <class Y>
static hipError_t dequantize_t(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds,
                               void* y, int64_t ldy, int M, int K, hipStream_t s) {
  const int units = (K + 7) / 8;
  const bool vec = ((reinterpret_cast<uintptr_t>(codes) | (uintptr_t)ldc) & 3) == 0 &&
                   ((reinterpret_cast<uintptr_t>(y) | (uintptr_t)(ldy * sizeof(Y))) & (8 * sizeof(Y) - 1)) == 0;
  return by_rows(M, units, [&](int64_t m, int rows) {
    const uint32_t total = (uint32_t)rows * (uint32_t)units;
    return launch_kernel(vec ? mx4_dequantize_kernel<Y, true> : mx4_dequantize_kernel<Y, false>,
                         groups_of(total), dim3(256), s, codes + m * ldc, ldc, scales + m * lds, lds,
                         static_cast<Y*>(y) + m * ldy, ldy, total, units, K);
  });
}

hipError_t launch_mx4_dequantize(const uint8_t* codes, int64_t ldc, const uint8_t* scales,
                                 int64_t lds, void* y, int y_dtype, int64_t ldy, int M, int K,
                                 hipStream_t s) {
  switch (y_dtype) {
    case XF16: return dequantize_t<_Float16>(codes, ldc, scales, lds, y, ldy, M, K, s);
    case XBF16: return dequantize_t<__bf16>(codes, ldc, scales, lds, y, ldy, M, K, s);
  }
  return dequantize_t<float>(codes, ldc, scales, lds, y, ldy, M, K, s);
}

hipError_t launch_mx4_pack(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds,
                           void* W, int batch, int N, int K, hipStream_t s) {
  const int strips = (N + 15) / 16;
  const int64_t all = (int64_t)batch * strips;
  const int64_t pieces = mx4_strip_bytes(K) / 16;
  const unsigned parts = (unsigned)(pieces > 256 * 64 ? 64 : (pieces + 255) / 256);
  const int64_t most = kMaxGroups / parts;
  hipError_t e = hipSuccess;
  for (int64_t f = 0; f < all && e == hipSuccess; f += most)
    e = launch_kernel(mx4_pack_kernel, dim3((unsigned)(all - f < most ? all - f : most), parts), dim3(256), s,
                      codes, ldc, scales, lds, static_cast<u32x4_t*>(W), strips, N, K, (int)f);
  return e;
}

}  // namespace qmm
