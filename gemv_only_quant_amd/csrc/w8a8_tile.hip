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
#include "w8a8_tile.h"

namespace qmm {

template <int KIND, int EPI, int MT, int NT, int DT>
__global__ __launch_bounds__(256) void tile_kernel(TileArgs g, int n_tiles, int m_tiles) {
  constexpr bool PAIR = EPI == EPI_GATED || EPI == EPI_GRAD;
  constexpr int BM = 16 * MT;
  constexpr int CPW = PAIR ? 8 * NT : 16 * NT;  // output columns per wave
  constexpr int UNITS = MT;                     // 16-byte chunks per thread and stage
  constexpr int EPI_WORDS = MT * epi_words(NT) + (EPI == EPI_GRAD ? epi_t_words(NT) : 0);
  constexpr int LDS_BYTES = 2 * BM * kStageBytes > 4 * EPI_WORDS * 4 ? 2 * BM * kStageBytes
                                                                     : 4 * EPI_WORDS * 4;
  __shared__ __align__(16) unsigned char lds[LDS_BYTES];
  __shared__ float sa[BM];
  u32x4_t(*xa)[BM * 16] = reinterpret_cast<u32x4_t(*)[BM * 16]>(lds);

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, quad = lane >> 4;
  int mt, nt;
  tile_of((int)blockIdx.x, n_tiles, m_tiles, &mt, &nt);
  const int m0 = mt * BM;
  const int n0 = (nt * 4 + wave) * CPW;  // this wave's first output column
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

  row_scales<EPI>(g, sa, m0, BM);

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
  Epilogue<KIND, EPI, NT, DT> epi;
  epi.init(g, n0, lane);
  epi.fetch(g, m0);
#pragma unroll
  for (int i = 0; i < MT; ++i) put_tile<KIND, NT>(acc[i], t0 + i * epi_words(NT), lane);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll 1
  for (int i = 0; i < MT; ++i)
    epi.tile(g, t0 + i * epi_words(NT), sa + 16 * i, t0 + MT * epi_words(NT), m0 + 16 * i,
             m0 + 16 * (i + 1));
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

// Whether 256-row tiles serve a product better: where they occupy a quarter of
// the CUs or more (codes, us, 256-row tiles / 64-row tiles: 512 x 4096 x 11008, 86
// tiles, 66 / 90; 333 x 1008 x 2777, 22 tiles, 28 / 18).
static bool many_rows(const TileArgs& t, int cols) {
  static const int want = env_int("QMM_TILE_LARGE");
  if (want >= 0 && t.splits <= 1) return want > 0;
  const int64_t tiles = (((int64_t)t.M + 255) / 256) * (((int64_t)t.N + cols - 1) / cols);
  return t.splits > 1 || tiles >= 64;
}

hipError_t launch_tile_scale(const TileArgs& t, hipStream_t s) {
  if (many_rows(t, 256)) return launch_large_scale(t, s);
  return launch_tile<kTypeI8, EPI_SCALE, 4, 4, XF16>(t, s);
}
hipError_t launch_tile_gated(const TileArgs& t, hipStream_t s) {
  if (many_rows(t, 128)) return launch_large_gated(t, s);
  return launch_tile<kTypeI8, EPI_GATED, 4, 4, XF16>(t, s);
}
hipError_t launch_tile_grad(const TileArgs& t, int dtype, hipStream_t s) {
  if (many_rows(t, 128)) return launch_large_grad(t, dtype, s);
  return dtype == XF16 ? launch_tile<kTypeI8, EPI_GRAD, 4, 4, XF16>(t, s)
                       : launch_tile<kTypeI8, EPI_GRAD, 4, 4, XBF16>(t, s);
}
hipError_t launch_tile_plain(const TileArgs& t, int dtype, hipStream_t s) {
  if (many_rows(t, 256)) return launch_large_plain(t, dtype, s);
  return dtype == XF16 ? launch_tile<XF16, EPI_PLAIN, 4, 4, XF16>(t, s)
                       : launch_tile<XBF16, EPI_PLAIN, 4, 4, XBF16>(t, s);
}

}  // namespace qmm
