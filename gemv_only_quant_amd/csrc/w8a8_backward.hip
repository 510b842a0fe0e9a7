// w8a8_backward.hip -- gradients of the int8 x int8 product and of the gated
// block on it.
//
//   dx[m, k] = sum_j D[m, j] W[j, k]       D  = dy sw c1 (gated: dg sg c1 | du su c1)
//   dW[n, k] = sum_m Dt[n, m] xq[m, k]     Dt = (dy sx c2)^t (gated: dg's, then du's)
//
// The right operands are the codes alone, as they lie in memory: they are exact
// in a 16-bit type, so each product has one rounding, that of D or Dt, and the
// product's kernel transposes and converts them on their way from LDS (a pass
// that wrote them transposed in 16 bits took 28 us for each 4096 x 11008, a tenth of the
// time at 4096 tokens and a quarter at 512).  c1 and c2 are the powers of two that
// bring the largest weight (token) scale to [1/2, 1): with scales of 1e-3 and fp16
// gradients the products would else lie among its subnormals.  They leave again,
// exactly, as the fp32 sums are stored.  bf16 has fp32's range: there both are 1, and
// neither the launch that finds them nor the factors are needed (4096 tokens: linear
// 11008 x 4096 692 -> 663 us, gated 4096 x 11008 1763 -> 1709).
//
// Steps: the powers of two (fp16, one workgroup); D and Dt -- from dy by scaling, or for
// the gated block by the gradient epilogue of the int8 product, which makes g and u
// again; then the two products.
#include <type_traits>

#include "w8a8_device.h"

namespace qmm {

// out[0..3] = c1, 1 / c1, c2, 1 / c2 with c a power of two, c max |scale| in
// [1/2, 1).  1 where the scales are all zero or not finite.
__global__ __launch_bounds__(1024) void scale_powers_kernel(const float* __restrict__ s0,
                                                            const float* __restrict__ s1,
                                                            const float* __restrict__ sx, int N,
                                                            int M, float* __restrict__ out) {
  __shared__ uint32_t part[2][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t top[2] = {0u, 0u};
  auto take = [&](const float* p, int n, uint32_t& t) {
    if (p == nullptr) return;
    // 8 loads in flight per thread, the last value again past the end (one at a
    // time 26112 scales take 13.9 us, so 6.8)
    for (int i0 = threadIdx.x; i0 < n; i0 += 8 * 1024) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = p[min(i0 + 1024 * j, n - 1)];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t b = __builtin_bit_cast(uint32_t, v[j]) & 0x7FFFFFFFu;
        if (b < 0x7F800000u && b > t) t = b;
      }
    }
  };
  take(s0, N, top[0]);
  take(s1, N, top[0]);
  take(sx, M, top[1]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
      const uint32_t o = (uint32_t)__shfl_xor((int)top[i], d);
      top[i] = o > top[i] ? o : top[i];
    }
    if (lane == 0) part[i][wave] = top[i];
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    const int i = threadIdx.x;
    uint32_t t = 0;
    for (int w = 0; w < 16; ++w) t = part[i][w] > t ? part[i][w] : t;
    // the exponent field e means [2^(e - 127), 2^(e - 126)); kept where both
    // powers are normal numbers
    int e = t == 0 ? 126 : (int)(t >> 23);
    e = e < 26 ? 26 : (e > 226 ? 226 : e);
    out[2 * i] = __builtin_bit_cast(float, (uint32_t)(253 - e) << 23);
    out[2 * i + 1] = __builtin_bit_cast(float, (uint32_t)(e + 1) << 23);
  }
}

// dy (M, N) -> d (M, Np) = dy sw c1 and, where dt is not NULL, dt (N, Mp) =
// (dy sx c2)^t, both with zeros where they only pad.  64 x 64 per workgroup,
// dt through LDS.
template <int DT>
__global__ __launch_bounds__(256) void scale_grad_kernel(
    const void* __restrict__ dy, int64_t lddy, const float* __restrict__ sw,
    const float* __restrict__ sx, const float* __restrict__ scal, void* __restrict__ d, int64_t Np,
    void* __restrict__ dt, int64_t Mp, int M, int N, int n_tiles) {
  typedef typename Half16<DT>::type T;
  typedef T T4 __attribute__((ext_vector_type(4)));
  typedef T T8 __attribute__((ext_vector_type(8)));
  __shared__ __align__(16) T t[64][72];
  const int n0 = (int)(blockIdx.x % (unsigned)n_tiles) * 64;
  const int m0 = (int)(blockIdx.x / (unsigned)n_tiles) * 64;
  const int tid = threadIdx.x;
  const T* src = static_cast<const T*>(dy);
  const bool vec = vec4_ok(dy, lddy, 2);
  const float c1 = DT == XF16 ? scal[0] : 1.f, c2 = DT == XF16 ? scal[2] : 1.f;
  const int col = 4 * (tid & 15), n = n0 + col;
  float s[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) s[j] = n + j < N ? sw[n + j] * c1 : 0.f;
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const int row = (tid >> 4) + 16 * h, m = m0 + row;
    float e[4] = {0.f, 0.f, 0.f, 0.f};
    if (m < M) {
      const T* p = src + (int64_t)m * lddy + n;
      if (vec && n + 4 <= N) {
        const T4 q = *reinterpret_cast<const T4*>(p);
#pragma unroll
        for (int j = 0; j < 4; ++j) e[j] = (float)q[j];
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n + j < N) e[j] = (float)p[j];
      }
      if (n < Np) {
        T4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = (T)(n + j < N ? e[j] * s[j] : 0.f);
        *reinterpret_cast<T4*>(static_cast<T*>(d) + (int64_t)m * Np + n) = o;
      }
    }
    if (dt != nullptr) {
      const float k = m < M ? sx[m] * c2 : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) t[col + j][row] = (T)(m < M ? e[j] * k : 0.f);
    }
  }
  if (dt == nullptr) return;
  __syncthreads();
  T* o = static_cast<T*>(dt);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = (tid >> 3) + 32 * h, r = 8 * (tid & 7);
    if (n0 + c < N && m0 + r < Mp)
      *reinterpret_cast<T8*>(o + (int64_t)(n0 + c) * Mp + m0 + r) =
          *reinterpret_cast<const T8*>(&t[c][r]);
  }
}

// Zeros rows of `len` elements of 2 or 4 bytes (a kernel, not a memset, so
// that the call can be captured in a HIP graph).
template <class T>
__global__ __launch_bounds__(256) void fill_zero_kernel(T* __restrict__ y, int64_t ld, int len,
                                                        int blocks_per_row) {
  const int64_t row = blockIdx.x / (unsigned)blocks_per_row;
  const int i = (int)(blockIdx.x % (unsigned)blocks_per_row) * 256 + (int)threadIdx.x;
  if (i < len) y[row * ld + i] = 0;
}

// ---------------------------------------------------------------- host side
hipError_t launch_fill_zero(void* y, int size, int64_t ld, int rows, int cols, hipStream_t s) {
  const int bpr = (cols + 255) / 256;
  const int64_t blocks = (int64_t)rows * bpr;
  if (blocks == 0) return hipSuccess;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  return size == 4 ? launch_kernel(fill_zero_kernel<uint32_t>, dim3((unsigned)blocks), dim3(256), s,
                                   static_cast<uint32_t*>(y), ld, cols, bpr)
                   : launch_kernel(fill_zero_kernel<uint16_t>, dim3((unsigned)blocks), dim3(256), s,
                                   static_cast<uint16_t*>(y), ld, cols, bpr);
}

BackwardPlan plan_backward(int M, int N, int K, bool gated, bool weight_grad) {
  BackwardPlan p{};
  const int64_t pad = kStageBytes / 2;  // 16-bit values
  p.parts = gated ? 2 : 1;
  p.Np = round_up(N, pad);
  p.Jp = p.parts * p.Np;
  p.Nr = round_up(N, 256);
  p.Mp = round_up(M, pad);
  size_t at = 256;  // scal at 0
  auto put = [&](int64_t elements) {
    const size_t here = at;
    at += (size_t)round_up(elements * 2, 256);
    return here;
  };
  p.d = put((int64_t)M * p.Jp);
  if (weight_grad) p.dt = put(p.parts * p.Nr * p.Mp);
  // fp32 sums of a product whose contraction is split; dx and dW in turn
  p.dx = plain_plan(M, K, 2 * p.Jp);
  p.dw = plain_plan(p.parts * p.Nr, K, 2 * p.Mp);
  const int64_t ld = round_up(K, 4);
  const int64_t px = p.dx.splits > 1 ? p.dx.splits * M * ld : 0;
  const int64_t pw = weight_grad && p.dw.splits > 1 ? p.dw.splits * p.parts * p.Nr * ld : 0;
  p.part = put(2 * (px > pw ? px : pw));
  p.bytes = at;
  return p;
}

template <int DT>
static hipError_t backward(const BackwardArgs& a, const BackwardPlan& p) {
  char* ws = static_cast<char*>(a.ws);
  float* scal = reinterpret_cast<float*>(ws + p.scal);
  const bool wgrad = a.dw[0] != nullptr;
  hipError_t e = hipSuccess;
  if (DT == XF16)
    e = launch_kernel(scale_powers_kernel, dim3(1), dim3(1024), a.stream, a.sw[0],
                      a.gated ? a.sw[1] : nullptr, wgrad ? a.sx : nullptr, a.N, a.M, scal);
  if (e != hipSuccess) return e;
  if (a.gated) {
    TileArgs t{};
    t.a = a.x;
    t.lda = a.ldx;
    t.b[0] = a.w[0], t.b[1] = a.w[1];
    t.ldb = a.ldw;
    t.M = a.M, t.N = a.N, t.kb = a.K;
    t.sa = a.sx;
    t.sb[0] = a.sw[0], t.sb[1] = a.sw[1];
    t.scal = scal;
    t.act = a.act;
    t.dh = a.dy;
    t.lddh = a.lddy;
    t.d = ws + p.d;
    t.dt = wgrad ? ws + p.dt : nullptr;
    t.Np = p.Np, t.Nr = p.Nr, t.Mp = p.Mp;
    e = launch_tile_grad(t, DT, a.stream);
  } else {
    const int n_tiles = (int)((p.Np + 63) / 64);
    const int64_t blocks = n_tiles * (((wgrad ? p.Mp : a.M) + 63) / 64);
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
    e = launch_kernel(scale_grad_kernel<DT>, dim3((unsigned)blocks), dim3(256), a.stream, a.dy,
                      a.lddy, a.sw[0], a.sx, scal, ws + p.d, p.Np, wgrad ? ws + p.dt : nullptr, p.Mp,
                      a.M, a.N, n_tiles);
  }
  if (e != hipSuccess) return e;

  TileArgs t{};  // dx
  t.a = ws + p.d;
  t.lda = 2 * p.Jp;
  t.b[0] = a.w[0], t.b[1] = a.w[1];
  t.ldb = a.ldw;
  t.brows = a.N, t.bpad = (int)p.Np;
  t.M = t.M2 = t.Mv = a.M;
  t.N = a.K;
  t.kb = (int)(2 * p.Jp);
  t.scal = scal + 1;
  t.part = reinterpret_cast<float*>(ws + p.part);
  t.plan = p.dx;
  t.y = a.dx;
  t.y_dtype = DT;
  t.ldy = a.lddx;
  e = launch_tile_plain(t, DT, a.stream);
  if (e != hipSuccess || !wgrad) return e;

  t.a = ws + p.dt;  // dW: rows 0 .. Nr of the first weight, then the second's
  t.lda = 2 * p.Mp;
  t.b[0] = a.x;
  t.ldb = a.ldx;
  t.brows = a.M, t.bpad = (int)p.Mp;
  t.M = (int)(p.parts * p.Nr);
  t.M2 = (int)p.Nr;
  t.Mv = a.N;
  t.kb = (int)(2 * p.Mp);
  t.scal = scal + 3;
  t.plan = p.dw;
  t.y = a.dw[0];
  t.y2 = a.dw[1];
  t.ldy = a.lddw;
  return launch_tile_plain(t, DT, a.stream);
}

hipError_t launch_backward(const BackwardArgs& a, const BackwardPlan& p) {
  return a.dtype == XF16 ? backward<XF16>(a, p) : backward<XBF16>(a, p);
}

}  // namespace qmm
