// w8a8_backward.hip -- gradients of the int8 x int8 product and of the gated
// block on it.
//
//   dx[m, k] = sum_j D[m, j] W[j, k]       D  = dy sw (gated: dg sg | du su)
//   dW[n, k] = sum_m Dt[n, m] xq[m, k]     Dt = (dy sx)^t (gated: dg's, then du's)
//
// The right operands are the codes alone, as they lie in memory: they are exact
// in a 16-bit type, so each product has one rounding, that of D or Dt, and the
// product's kernel transposes and converts them on their way from LDS (a pass
// that wrote them transposed in 16 bits took 28 us for each 4096 x 11008, a tenth of the
// time at 4096 tokens and a quarter at 512).
//
// bf16 has fp32's range.  An fp16 D or Dt of plain values would not do: their products of
// a gradient and a scale reach from below its subnormals to beyond its largest value, and
// rows of one operand lie decades apart.  There each row has a power of two of its own,
// by its largest value, which leaves again, exactly, as the fp32 sums are stored.  The
// kernels that make the operands know no more of a row than a block; they take the
// block's power and note it as a level, and a second launch brings a row's blocks to one
// level.  What this costs beside one power for all rows, found from the scales alone (which
// loses such rows, and dg beyond 65504): dx 512 x 11008 x 4096 73.4 -> 74.3 us, both gradients
// 4096 x 11008 x 4096 689 -> 698; gated, dx 509 x 4096 x 11008 185 -> 185, all three at 64
// tokens 115 -> 122, at 4096 1720 -> 1780.
//
// Steps: D and Dt -- from dy by scaling, or for the gated block by the gradient epilogue
// of the int8 product, which makes g and u again; their levels (fp16); then the two
// products.
#include <type_traits>

#include "w8a8_device.h"

namespace qmm {

// dy (M, N) -> d (M, Np) = dy sw and, where dt is not NULL, dt (N, Mp) = (dy sx)^t,
// both with zeros where they only pad; in fp16 each block times its power of two, whose
// levels go to de and dte.  64 x 64 per workgroup, dt through LDS.  A wave has 16 rows,
// 4 at a time, 16 lanes to a row.
template <int DT>
__global__ __launch_bounds__(256) void scale_grad_kernel(
    const void* __restrict__ dy, int64_t lddy, const float* __restrict__ sw,
    const float* __restrict__ sx, void* __restrict__ d, int64_t Np, void* __restrict__ dt,
    int64_t Mp, uint8_t* __restrict__ de, uint8_t* __restrict__ dte, int M, int N, int n_tiles,
    int m_first) {
  typedef typename Half16<DT>::type T;
  typedef T T4 __attribute__((ext_vector_type(4)));
  typedef T T8 __attribute__((ext_vector_type(8)));
  __shared__ __align__(16) T t[64][72];
  const int n0 = (int)(blockIdx.x % (unsigned)n_tiles) * 64;
  const int m0 = m_first + (int)(blockIdx.x / (unsigned)n_tiles) * 64;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const T* src = static_cast<const T*>(dy);
  const bool vec = vec4_ok(dy, lddy, 2);
  const int col = 4 * (lane & 15), n = n0 + col;
  auto row_of = [&](int h) { return 16 * wave + 4 * h + (lane >> 4); };
  float s[4], e[4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) s[j] = n + j < N ? sw[n + j] : 0.f;
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const int m = m0 + row_of(h);
#pragma unroll
    for (int j = 0; j < 4; ++j) e[h][j] = 0.f;
    if (m >= M) continue;
    const T* p = src + (int64_t)m * lddy + n;
    if (vec && n + 4 <= N) {
      const T4 q = *reinterpret_cast<const T4*>(p);
#pragma unroll
      for (int j = 0; j < 4; ++j) e[h][j] = (float)q[j];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j < N) e[h][j] = (float)p[j];
    }
  }
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const int m = m0 + row_of(h);
    float v[4], k = 1.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = n + j < N ? e[h][j] * s[j] : 0.f;
    if constexpr (DT == XF16) {
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) top = fmaxf(top, fabsf(v[j]));
      const uint32_t level = level_of(lanes_max<8>(top));
      k = level_power(level);
      if ((lane & 7) == 0 && m < M) de[(int64_t)m * (Np / kLevelD) + n / kLevelD] = (uint8_t)level;
    }
    T4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = (T)(v[j] * k);
    if (m < M) *reinterpret_cast<T4*>(static_cast<T*>(d) + (int64_t)m * Np + n) = o;
  }
  if (dt == nullptr) return;
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const int m = m0 + row_of(h);
    const float k = m < M ? sx[m] : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) e[h][j] = m < M ? e[h][j] * k : 0.f;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float k = 1.f;
    if constexpr (DT == XF16) {
      float top = 0.f;
#pragma unroll
      for (int h = 0; h < 4; ++h) top = fmaxf(top, fabsf(e[h][j]));
      const uint32_t level = level_of(rows4_max(top));
      k = level_power(level);
      if (lane < 16 && n + j < N)
        dte[(int64_t)(n + j) * (Mp / kLevelT) + m0 / kLevelT + wave] = (uint8_t)level;
    }
#pragma unroll
    for (int h = 0; h < 4; ++h) t[col + j][row_of(h)] = (T)(e[h][j] * k);
  }
  __syncthreads();
  T* o = static_cast<T*>(dt);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = (tid >> 3) + 32 * h, r = 8 * (tid & 7);
    if (n0 + c < N)
      *reinterpret_cast<T8*>(o + (int64_t)(n0 + c) * Mp + m0 + r) =
          *reinterpret_cast<const T8*>(&t[c][r]);
  }
}

// The rows of an fp16 operand brought to one level each, the largest of their blocks':
// blocks of a lower one are multiplied by what is missing, down from where they are
// exact to where they lose less than 2^-31 of the row's largest value.  inv: what a
// product with the row is multiplied by afterwards.
struct LevelRows {
  _Float16* d;        // `parts` of `len` columns, each with the same levels
  const uint8_t* e;   // (rows, len / (8 << shift))
  float* inv;
  int64_t ld;
  int rows, len, parts, shift;
  int live, pitch;    // rows that exist of each `pitch`
  int waves;          // 1 or 4 to a row
  int blocks;
};

__global__ __launch_bounds__(256) void level_rows_kernel(LevelRows a, LevelRows b) {
  __shared__ uint32_t part[4];
  const bool second = (int)blockIdx.x >= a.blocks;
  const LevelRows& g = second ? b : a;
  const int block = (int)blockIdx.x - (second ? a.blocks : 0);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int i = g.waves == 4 ? block : 4 * block + wave;
  const bool live = i < g.rows;
  const int row = live ? i / g.live * g.pitch + i % g.live : 0;
  const int t = g.waves == 4 ? (int)threadIdx.x : lane, step = 64 * g.waves;
  const int vectors = g.len / 8, levels = vectors >> g.shift;
  const uint8_t* e = g.e + (int64_t)row * levels;
  uint32_t top = 0;
  for (int l = t; l < levels; l += step) top = e[l] > top ? e[l] : top;
  top = wave_max_u32(top);
  if (g.waves == 4) {
    if (lane == 0) part[wave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) top = part[w] > top ? part[w] : top;
  }
  if (!live) return;
  if (t == 0) g.inv[row] = level_inverse(top);
  // 16 bytes per lane, 4 loads in flight; blocks that stay are loaded from nowhere
  for (int p = 0; p < g.parts; ++p) {
    _Float16* d = g.d + (int64_t)row * g.ld + (int64_t)p * g.len;
    const buf_t buf = make_buf(d, (uint32_t)g.len * 2);
    for (int v0 = t; v0 < vectors; v0 += 4 * step) {
      uint32_t down[4];
      u32x4_t x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int v = v0 + j * step;
        down[j] = v < vectors ? top - e[v >> g.shift] : 0u;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = buf_load128(buf, down[j] != 0 ? 16 * (v0 + j * step) : 0x60000000);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (down[j] == 0) continue;
        // (an infinity's row: the finite rest may vanish, but meets no infinite factor)
        const float k = __builtin_bit_cast(float, (127u - (down[j] < 120u ? down[j] : 120u)) << 23);
        typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
        half8_t h = __builtin_bit_cast(half8_t, x[j]);
#pragma unroll
        for (int c = 0; c < 8; ++c) h[c] = (_Float16)((float)h[c] * k);
        *reinterpret_cast<half8_t*>(d + 8 * (v0 + j * step)) = h;
      }
    }
  }
}

// Zeros rows of `len` elements of 2 or 4 bytes, 256 of one row at a time (a kernel, not a
// memset, so that the call can be captured in a HIP graph).
template <class T>
__global__ __launch_bounds__(256) void fill_zero_kernel(T* __restrict__ y, int64_t ld, int len,
                                                        int blocks_per_row, int64_t blocks) {
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    const int i = (int)(b % blocks_per_row) * 256 + (int)threadIdx.x;
    if (i < len) y[b / blocks_per_row * ld + i] = 0;
  }
}

// ---------------------------------------------------------------- host side
hipError_t launch_fill_zero(void* y, int size, int64_t ld, int rows, int cols, hipStream_t s) {
  const int bpr = (cols + 255) / 256;
  const int64_t blocks = (int64_t)rows * bpr;
  if (blocks == 0) return hipSuccess;
  const dim3 grid((unsigned)(blocks < kMaxGroups ? blocks : kMaxGroups));
  return size == 4 ? launch_kernel(fill_zero_kernel<uint32_t>, grid, dim3(256), s,
                                   static_cast<uint32_t*>(y), ld, cols, bpr, blocks)
                   : launch_kernel(fill_zero_kernel<uint16_t>, grid, dim3(256), s,
                                   static_cast<uint16_t*>(y), ld, cols, bpr, blocks);
}

BackwardPlan plan_backward(int M, int N, int K, bool gated, bool weight_grad) {
  BackwardPlan p{};
  const int64_t pad = kStageBytes / 2;  // 16-bit values
  p.parts = gated ? 2 : 1;
  p.Np = round_up(N, pad);
  p.Jp = p.parts * p.Np;
  p.Nr = round_up(N, 256);
  p.Mp = round_up(M, pad);
  size_t at = 0;
  auto put = [&](int64_t elements) {
    const size_t here = at;
    at += (size_t)round_up(elements * 2, 256);
    return here;
  };
  p.d = put((int64_t)M * p.Jp);
  p.de = put(((int64_t)M * (p.Np / kLevelD) + 1) / 2);
  p.inv = put(2 * (int64_t)M);
  if (weight_grad) {
    p.dt = put(p.parts * p.Nr * p.Mp);
    p.dte = put(p.parts * p.Nr * (p.Mp / kLevelT) / 2);
    p.invt = put(2 * p.parts * p.Nr);
  }
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

// Both operands' rows to one level each.  Four waves to a row of more than 2048 values.
static hipError_t level_operands(const BackwardArgs& a, const BackwardPlan& p, char* ws) {
  auto rows = [&](size_t d, size_t e, size_t inv, int64_t n, int64_t len, int parts, int shift) {
    LevelRows r{};
    r.d = reinterpret_cast<_Float16*>(ws + d);
    r.e = reinterpret_cast<const uint8_t*>(ws + e);
    r.inv = reinterpret_cast<float*>(ws + inv);
    r.ld = parts * len;
    r.rows = r.live = r.pitch = (int)n;
    r.len = (int)len, r.parts = parts, r.shift = shift;
    r.waves = parts * len > 2048 ? 4 : 1;
    r.blocks = (r.rows * r.waves + 3) / 4;
    return r;
  };
  LevelRows x = rows(p.d, p.de, p.inv, a.M, p.Np, p.parts, 2), w{};
  if (a.dw[0] != nullptr) {
    w = rows(p.dt, p.dte, p.invt, (int64_t)p.parts * a.N, p.Mp, 1, 1);
    w.live = a.N, w.pitch = (int)p.Nr;
  }
  return launch_kernel(level_rows_kernel, dim3((unsigned)(x.blocks + w.blocks)), dim3(256), a.stream, x, w);
}

template <int DT>
static hipError_t backward(const BackwardArgs& a, const BackwardPlan& p) {
  char* ws = static_cast<char*>(a.ws);
  const bool wgrad = a.dw[0] != nullptr;
  uint8_t* de = reinterpret_cast<uint8_t*>(ws + p.de);
  uint8_t* dte = wgrad ? reinterpret_cast<uint8_t*>(ws + p.dte) : nullptr;
  hipError_t e;
  if (a.gated) {
    TileArgs t{};
    t.a = a.x;
    t.lda = a.ldx;
    t.b[0] = a.w[0], t.b[1] = a.w[1];
    t.ldb = a.ldw;
    t.M = a.M, t.N = a.N, t.kb = a.K;
    t.sa = a.sx;
    t.sb[0] = a.sw[0], t.sb[1] = a.sw[1];
    t.act = a.act;
    t.dh = a.dy;
    t.lddh = a.lddy;
    t.d = ws + p.d;
    t.dt = wgrad ? ws + p.dt : nullptr;
    t.de = de, t.dte = dte;
    t.Np = p.Np, t.Nr = p.Nr, t.Mp = p.Mp;
    e = launch_tile_grad(t, DT, a.stream);
  } else {
    const int n_tiles = (int)(p.Np / 64);
    const int64_t m_tiles = ((wgrad ? p.Mp : a.M) + 63) / 64, most = kMaxGroups / n_tiles;
    e = hipSuccess;
    for (int64_t m = 0; m < m_tiles && e == hipSuccess; m += most) {
      const int64_t blocks = n_tiles * (m_tiles - m < most ? m_tiles - m : most);
      e = launch_kernel(scale_grad_kernel<DT>, dim3((unsigned)blocks), dim3(256), a.stream, a.dy, a.lddy,
                        a.sw[0], a.sx, ws + p.d, p.Np, wgrad ? ws + p.dt : nullptr, p.Mp, de, dte, a.M,
                        a.N, n_tiles, (int)(64 * m));
    }
  }
  if (e != hipSuccess) return e;
  if (DT == XF16) e = level_operands(a, p, ws);
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
  t.sa = reinterpret_cast<const float*>(ws + p.inv);
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
  t.sa = reinterpret_cast<const float*>(ws + p.invt);
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
