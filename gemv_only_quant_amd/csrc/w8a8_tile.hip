// w8a8_tile.hip -- C = A B^t on the matrix cores for int8 codes
// (v_mfma_i32_16x16x64_i8, exact sums) and for 16-bit operands
// (v_mfma_f32_16x16x32_{f16,bf16}), with the epilogues of the int8 x int8
// operators:
//   SCALE  y = C sa[m] sb[n]
//   GATED  h = act(g) u for two products g, u of the same left operand
//   GRAD   dg = dh u act'(g), du = dh act(g), left as 16-bit operands of the
//          gradients' products, once row-major and once transposed
//   PLAIN  y = C * (a power of two), 16-bit
//
// Both operands have the contracted axis contiguous, and one 16-byte chunk
// per lane is one operand of either kind of MFMA (16 int8 or 8 16-bit
// values), so one kernel moves bytes and only the instruction differs.
// A workgroup covers 16 MT rows x 4 waves x NT strips of 16 columns; a stage
// is 256 contracted bytes.  A goes through LDS (chunk c of row r at slot
// 16 r + (c ^ r): conflict-free operand reads), shared by the 4 waves; each
// wave reads its own columns of B straight into operands.
#include <type_traits>

#include "w8a8_device.h"

namespace qmm {

enum { EPI_SCALE = 0, EPI_GATED = 1, EPI_GRAD = 2, EPI_PLAIN = 3 };

// KIND: kTypeI8, XF16 or XBF16
template <int KIND> struct Acc { typedef f32x4_t type; };
template <> struct Acc<kTypeI8> { typedef i32x4_t type; };

template <int KIND>
__device__ __forceinline__ typename Acc<KIND>::type mfma_t(const u32x4_t& a, const u32x4_t& b,
                                                           typename Acc<KIND>::type c) {
  if constexpr (KIND == kTypeI8)
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a),
                                                 __builtin_bit_cast(i32x4_t, b), c, 0, 0, 0);
  else if constexpr (KIND == XF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                  __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// One 16-row tile of a wave (accumulators of its NT strips) through LDS to
// the epilogue: rows of 4 consecutive columns per lane.  `t0` is the tile's
// LDS (16 rows of 16 NT + 4 words), n0 the wave's first output column, m0
// the tile's first row.
template <int KIND, int EPI, int NT, int DT>
__device__ __forceinline__ void finish_tile(const TileArgs& g, const typename Acc<KIND>::type (&acc)[NT],
                                            uint32_t* t0, int m0, int n0, int lane) {
  constexpr bool PAIR = EPI == EPI_GATED || EPI == EPI_GRAD;
  constexpr int COLS = PAIR ? 8 * NT : 16 * NT;  // output columns of the wave
  constexpr int LDT = 16 * NT + 4;
  constexpr int LPR = COLS / 4;     // lanes per row
  constexpr int RPP = 64 / LPR;     // rows per pass
  const int l16 = lane & 15, quad = lane >> 4;
#pragma unroll
  for (int s = 0; s < NT; ++s)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      // through a value: a bit cast of the vector's element itself takes
      // element 0 whatever r is, with this compiler
      const auto e = acc[s][r];
      t0[(4 * quad + r) * LDT + 16 * s + l16] = __builtin_bit_cast(uint32_t, e);
    }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  const int col = 4 * (lane % LPR), n = n0 + col;
  const int nn = min(4, g.N - n);  // columns of this lane that exist (may be <= 0)
  typedef typename Acc<KIND>::type acc_t;

  if constexpr (EPI == EPI_SCALE || EPI == EPI_PLAIN) {
    float sb[4] = {1.f, 1.f, 1.f, 1.f};
    if constexpr (EPI == EPI_SCALE) {
#pragma unroll
      for (int j = 0; j < 4; ++j) sb[j] = j < nn ? g.sb[0][n + j] : 0.f;
    }
    with_y(g.y, g.y_dtype, [&](auto* yt) {
      typedef typename std::remove_pointer<decltype(yt)>::type T;
      const bool vec = vec4_ok(yt, g.ldy, (int)sizeof(T));
#pragma unroll
      for (int p = 0; p < 16 / RPP; ++p) {
        const int row = RPP * p + lane / LPR, m = m0 + row;
        const acc_t c = *reinterpret_cast<const acc_t*>(t0 + row * LDT + col);
        if (m >= g.M || nn <= 0) continue;
        float v[4];
        if constexpr (EPI == EPI_SCALE) {
          const float sa = g.sa[m];
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = (float)c[j] * (sa * sb[j]);
          store4(yt + (int64_t)m * g.ldy + n, v, nn, vec);
        } else {
          const float k = *g.scal;
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = c[j] * k;
          const bool second = m >= g.M2;
          const int mo = second ? m - g.M2 : m;
          if (mo < g.Mv) {
            T* yo = second ? static_cast<T*>(g.y2) : yt;
            store4(yo + (int64_t)mo * g.ldy + n, v, nn, vec);
          }
        }
      }
    });
  } else {
    float sg[4], su[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sg[j] = j < nn ? g.sb[0][n + j] : 0.f;
      su[j] = j < nn ? g.sb[1][n + j] : 0.f;
    }
    if constexpr (EPI == EPI_GATED) {
      with_y(g.y, g.y_dtype, [&](auto* yt) {
        typedef typename std::remove_pointer<decltype(yt)>::type T;
        const bool vec = vec4_ok(yt, g.ldy, (int)sizeof(T));
#pragma unroll
        for (int p = 0; p < 16 / RPP; ++p) {
          const int row = RPP * p + lane / LPR, m = m0 + row;
          const acc_t cg = *reinterpret_cast<const acc_t*>(t0 + row * LDT + col);
          const acc_t cu = *reinterpret_cast<const acc_t*>(t0 + row * LDT + COLS + col);
          if (m >= g.M || nn <= 0) continue;
          const float sa = g.sa[m];
          float v[4], d;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            v[j] = act_parts(g.act, (float)cg[j] * (sa * sg[j]), &d) * ((float)cu[j] * (sa * su[j]));
          store4(yt + (int64_t)m * g.ldy + n, v, nn, vec);
        }
      });
    } else {
      // dg and du in fp32, then d = (dg sg c1 | du su c1) row-major and
      // dt = (dg sx c2 | du sx c2) transposed through LDS, zeros where a row
      // or column only pads
      typedef typename Half16<DT>::type T;
      typedef T T4 __attribute__((ext_vector_type(4)));
      typedef T T8 __attribute__((ext_vector_type(8)));
      constexpr int LDH = 24;  // 16 rows of a column, padded to keep 16-byte reads aligned
      T* tt = reinterpret_cast<T*>(t0 + 16 * LDT);
      const float c1 = g.scal[0], c2 = g.scal[2];
      const T* dh = static_cast<const T*>(g.dh);
      T* dd = static_cast<T*>(g.d);
      const bool vec = vec4_ok(dh, g.lddh, 2);
#pragma unroll
      for (int p = 0; p < 16 / RPP; ++p) {
        const int row = RPP * p + lane / LPR, m = m0 + row;
        const acc_t cg = *reinterpret_cast<const acc_t*>(t0 + row * LDT + col);
        const acc_t cu = *reinterpret_cast<const acc_t*>(t0 + row * LDT + COLS + col);
        T4 dgv = {}, duv = {};
        T tg[4] = {}, tu[4] = {};
        if (m < g.M && nn > 0) {
          const T* src = dh + (int64_t)m * g.lddh + n;
          float e[4];
          if (vec && nn >= 4) {
            const T4 q = *reinterpret_cast<const T4*>(src);
#pragma unroll
            for (int j = 0; j < 4; ++j) e[j] = (float)q[j];
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) e[j] = j < nn ? (float)src[j] : 0.f;
          }
          const float sa = g.sa[m];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j >= nn) continue;
            const float gv = (float)cg[j] * (sa * sg[j]), uv = (float)cu[j] * (sa * su[j]);
            float da;
            const float a = act_parts(g.act, gv, &da);
            const float dg = e[j] * uv * da, du = e[j] * a;
            dgv[j] = (T)(dg * (sg[j] * c1));
            duv[j] = (T)(du * (su[j] * c1));
            tg[j] = (T)(dg * (sa * c2));
            tu[j] = (T)(du * (sa * c2));
          }
        }
        if (m < g.M && n < g.Np) {  // n is a multiple of 4 and Np of 128
          T* o = dd + (int64_t)m * (2 * g.Np) + n;
          *reinterpret_cast<T4*>(o) = dgv;
          *reinterpret_cast<T4*>(o + g.Np) = duv;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          tt[(col + j) * LDH + row] = tg[j];
          tt[(COLS + col + j) * LDH + row] = tu[j];
        }
      }
      if (g.dt != nullptr && m0 < g.Mp) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        T* dt = static_cast<T*>(g.dt);
        for (int c = lane; c < 2 * COLS; c += 64) {
          const int cn = n0 + c % COLS;
          if (cn >= g.N) continue;
          const T8 a = *reinterpret_cast<const T8*>(tt + c * LDH);
          const T8 b = *reinterpret_cast<const T8*>(tt + c * LDH + 8);
          T* o = dt + ((int64_t)(c / COLS) * g.Nr + cn) * g.Mp + m0;
          *reinterpret_cast<T8*>(o) = a;
          *reinterpret_cast<T8*>(o + 8) = b;
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      }
    }
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}

template <int KIND, int EPI, int MT, int NT, int DT>
__global__ __launch_bounds__(256) void tile_kernel(TileArgs g, int n_tiles, int m_tiles) {
  constexpr bool PAIR = EPI == EPI_GATED || EPI == EPI_GRAD;
  constexpr int BM = 16 * MT;
  constexpr int CPW = PAIR ? 8 * NT : 16 * NT;  // output columns per wave
  constexpr int UNITS = MT;                     // 16-byte chunks per thread and stage
  constexpr int EPI_WORDS = 16 * (16 * NT + 4) + (EPI == EPI_GRAD ? 16 * NT * 24 / 2 : 0);
  constexpr int LDS_BYTES = 2 * BM * kStageBytes > 4 * EPI_WORDS * 4 ? 2 * BM * kStageBytes
                                                                     : 4 * EPI_WORDS * 4;
  __shared__ __align__(16) unsigned char lds[LDS_BYTES];
  u32x4_t(*xa)[BM * 16] = reinterpret_cast<u32x4_t(*)[BM * 16]>(lds);

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, quad = lane >> 4;
  const int w = xcd_remap((int)blockIdx.x, n_tiles * m_tiles);
  const int m0 = (w / n_tiles) * BM;
  const int n0 = ((w % n_tiles) * 4 + wave) * CPW;  // this wave's first output column
  const int kb = g.kb, nst = (kb + kStageBytes - 1) / kStageBytes;
  const int kb16 = (kb + 15) & ~15;

  // descriptors end with the operand's last row (chunks past it read zeros)
  const int rows = min(BM, g.M - m0);  // none where the tile only pads
  const buf_t ab = make_buf(static_cast<const char*>(g.a) + (int64_t)m0 * g.lda,
                            rows > 0 ? (uint32_t)((rows - 1) * g.lda + kb16) : 0u);
  const int nc0 = min(n0, g.N - 1);
  const int bcols = min(CPW, g.N - nc0);
  const uint32_t brange = (uint32_t)((bcols - 1) * g.ldb + kb16);
  buf_t bb[2];
#pragma unroll
  for (int i = 0; i < (PAIR ? 2 : 1); ++i)
    bb[i] = make_buf(static_cast<const char*>(g.b[i]) + (int64_t)nc0 * g.ldb, brange);

  typedef typename Acc<KIND>::type acc_t;
  acc_t acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int s = 0; s < NT; ++s) acc[i][s] = acc_t{0, 0, 0, 0};

  // chunk u of this thread: row (tid + 256 u) / 16, chunk column tid % 16
  const int crow = (int)threadIdx.x >> 4, ccol = (int)threadIdx.x & 15;
  u32x4_t xr[UNITS], br[NT][4];
  auto load = [&](int st) {
    const int k = st * kStageBytes;
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const int kk = k + 16 * ccol;
      xr[u] = buf_load128(ab, kk < kb ? (crow + 16 * u) * (int)g.lda + kk : -16);
      if (KIND == kTypeI8) xr[u] = clear_tail(xr[u], kk, kb);
    }
#pragma unroll
    for (int s = 0; s < NT; ++s) {
      const int row = (PAIR ? 16 * (s % (NT / 2)) : 16 * s) + l16;
      const buf_t b = bb[PAIR ? s / (NT / 2) : 0];
#pragma unroll
      for (int j = 0; j < 4; ++j) br[s][j] = buf_load128(b, row * (int)g.ldb + k + 64 * j + 16 * quad);
    }
  };
  if (nst > 0) load(0);
  for (int st = 0; st < nst; ++st) {
    u32x4_t* buf = xa[st & 1];
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const int row = crow + 16 * u;
      buf[16 * row + (ccol ^ (row & 15))] = xr[u];
    }
    u32x4_t b[NT][4];
#pragma unroll
    for (int s = 0; s < NT; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j) b[s][j] = br[s][j];
    __syncthreads();
    if (st + 1 < nst) load(st + 1);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const u32x4_t a = buf[256 * i + 16 * l16 + ((4 * j + quad) ^ l16)];
#pragma unroll
        for (int s = 0; s < NT; ++s) acc[i][s] = mfma_t<KIND>(a, b[s][j], acc[i][s]);
      }
  }
  __syncthreads();  // the stages' LDS becomes the epilogue's

  uint32_t* t0 = reinterpret_cast<uint32_t*>(lds) + wave * EPI_WORDS;
#pragma unroll
  for (int i = 0; i < MT; ++i)
    finish_tile<KIND, EPI, NT, DT>(g, acc[i], t0, m0 + 16 * i, n0, lane);
}

// ---------------------------------------------------------------- host side
template <int KIND, int EPI, int MT, int NT, int DT>
static hipError_t launch_tile(const TileArgs& t, hipStream_t s) {
  constexpr int cpg = 4 * (EPI == EPI_GATED || EPI == EPI_GRAD ? 8 : 16) * NT;
  // the gradient epilogue also writes the padding of its operands
  const int64_t cols = EPI == EPI_GRAD ? t.Np : t.N;
  const int64_t rows = EPI == EPI_GRAD && t.dt != nullptr ? t.Mp : t.M;
  const int64_t n_tiles = (cols + cpg - 1) / cpg, m_tiles = (rows + 16 * MT - 1) / (16 * MT);
  if (n_tiles * m_tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
  return launch_kernel(tile_kernel<KIND, EPI, MT, NT, DT>, dim3((unsigned)(n_tiles * m_tiles)),
                       dim3(256), s, t, (int)n_tiles, (int)m_tiles);
}

hipError_t launch_tile_scale(const TileArgs& t, hipStream_t s) {
  return launch_tile<kTypeI8, EPI_SCALE, 4, 4, XF16>(t, s);
}
hipError_t launch_tile_gated(const TileArgs& t, hipStream_t s) {
  return launch_tile<kTypeI8, EPI_GATED, 4, 4, XF16>(t, s);
}
hipError_t launch_tile_grad(const TileArgs& t, int dtype, hipStream_t s) {
  return dtype == XF16 ? launch_tile<kTypeI8, EPI_GRAD, 4, 4, XF16>(t, s)
                       : launch_tile<kTypeI8, EPI_GRAD, 4, 4, XBF16>(t, s);
}
hipError_t launch_tile_plain(const TileArgs& t, int dtype, hipStream_t s) {
  return dtype == XF16 ? launch_tile<XF16, EPI_PLAIN, 4, 4, XF16>(t, s)
                       : launch_tile<XBF16, EPI_PLAIN, 4, 4, XBF16>(t, s);
}

}  // namespace qmm
