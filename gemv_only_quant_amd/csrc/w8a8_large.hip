// w8a8_large.hip -- the products of w8a8_tile.hip for many rows: 256-row
// tiles, bound by the matrix cores.
//
//  * workgroup tile 256 rows x 4 waves x 64 columns of B, one workgroup per
//    CU; a wave owns all 256 rows x 4 strips = 16 x 4 MFMA tiles, 256
//    accumulators per lane pinned to the matrix-core (AGPR) registers;
//  * a stage is 256 contracted bytes (256 int8 or 128 16-bit values).  The A
//    tile of a stage, 64 KiB, is shared by the waves through double-buffered
//    LDS, filled by buffer loads straight to LDS in the swizzled row layout
//    (chunk c of row r at slot 16 r + (c ^ r): whole 256-byte rows per load,
//    conflict-free ds_read_b128 operands).  At 4 MFMAs per operand read the
//    LDS is busy for 5/8 of the MFMAs' time; with B in LDS too it would be the bound;
//  * each wave reads its own columns of B straight into operands, a stage
//    ahead in a second set of registers, so nothing inside a stage waits for
//    memory: the loads of the next stage go out in the first half of this one
//    and are waited for at its end.
// Every address is in the offset that the buffer's range is checked against:
// rows past M and columns past N read zeros.
#include "w8a8_tile.h"

namespace qmm {

constexpr int kBigMT = 16;  // 16-row tiles per workgroup
static constexpr int kWaitVm0Big = 0x0F70;  // s_waitcnt vmcnt(0), other counters at maximum

// MFMA with its accumulator pinned to the AGPRs (left to itself the register
// allocator moves 256 live accumulators between the register files).
template <int KIND>
__device__ __forceinline__ void mfma_pinned(typename Acc<KIND>::type& c, const u32x4_t& a,
                                            const u32x4_t& b) {
  if constexpr (KIND == kTypeI8)
    asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
  else if constexpr (KIND == XF16)
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
  else
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}

// LDS of a workgroup in 16-byte words: two stages of A, then half of the row
// tiles at a time for the epilogue (4 waves of as many words each).
template <int EPI, int NT> struct LargeLds {
  static constexpr int EPI_WORDS =
      (kBigMT / 2) * epi_words(NT) + (EPI == EPI_GRAD ? epi_t_words(NT) : 0);
  static constexpr int STAGES = 2 * 16 * kBigMT * 16;
  static constexpr int SCALES = STAGES > EPI_WORDS ? STAGES : EPI_WORDS;  // where the row scales lie
  static constexpr int WORDS16 = SCALES + 16 * kBigMT / 4;
};

// (a device function beside its kernel: the host pass drops a kernel whose own
// body has matrix-core registers in inline asm)
template <int KIND, int EPI, int NT, int DT>
__device__ __forceinline__ void large_body(const TileArgs& g, int n_tiles, int m_tiles,
                                           u32x4_t* lds) {
  constexpr bool PAIR = EPI == EPI_GATED || EPI == EPI_GRAD;
  constexpr int MT = kBigMT, BM = 16 * MT, STEPS = kStageBytes / 64;
  constexpr int CPW = PAIR ? 8 * NT : 16 * NT;  // output columns per wave
  constexpr int EPI_WORDS = LargeLds<EPI, NT>::EPI_WORDS;
  u32x4_t(*xa)[BM * 16] = reinterpret_cast<u32x4_t(*)[BM * 16]>(lds);

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, quad = lane >> 4;
  int mt, nt;
  tile_of((int)blockIdx.x, n_tiles, m_tiles, &mt, &nt);
  const int m0 = mt * BM;
  const int n0 = (nt * 4 + wave) * CPW;
  const int kb = g.kb, nst = (kb + kStageBytes - 1) / kStageBytes;
  const int kb16 = (kb + 15) & ~15;
  const int lda = (int)g.lda, ldb = (int)g.ldb;

  // One buffer per 16 rows of A that this wave moves and per strip of B that it
  // reads, from a stage's first byte to the end of the last row: the lanes'
  // offsets are then the same few registers for all of them.
  struct Rows {
    const char* base;
    int range;  // bytes, 0 where no row exists
  };
  auto rows_of = [&](const void* p, int64_t ld, int first, int count, int limit) {
    const int n = min(count, limit - first);
    Rows r;
    r.base = static_cast<const char*>(p) + (int64_t)(n > 0 ? first : 0) * ld;
    r.range = n > 0 ? (int)((n - 1) * ld) + kb16 : 0;
    return r;
  };
  auto at_stage = [&](const Rows& r, int st) {
    return make_buf(r.base + st * kStageBytes, r.range > 0 ? (uint32_t)(r.range - st * kStageBytes) : 0u);
  };
  Rows ar_[4], br_[NT];
#pragma unroll
  for (int i = 0; i < 4; ++i) ar_[i] = rows_of(g.a, g.lda, m0 + 64 * wave + 16 * i, 16, g.M);
#pragma unroll
  for (int s = 0; s < NT; ++s)
    br_[s] = PAIR ? rows_of(g.b[s / (NT / 2)], g.ldb, n0 + 16 * (s % (NT / 2)), 16, g.N)
                  : rows_of(g.b[0], g.ldb, n0 + 16 * s, 16, g.N);

  // A: load unit f (1 KiB) is rows 4 (f % 4) .. + 3 of row tile f / 4; lane p's
  // 16 bytes land at slot 64 (f % 4) + p of the tile, so it fetches chunk (p %
  // 16) ^ r of row r = 4 (f % 4) + p / 16.  Wave w moves units 16 w .. + 15.
  int xo[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) xo[c] = (4 * c + quad) * lda + 16 * (l16 ^ (4 * c + quad));
  const int bo = l16 * ldb + 16 * quad;

  float* sa = reinterpret_cast<float*>(lds + LargeLds<EPI, NT>::SCALES);
  row_scales<EPI>(g, sa, m0, BM);

  typedef typename Acc<KIND>::type acc_t;
  acc_t acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int s = 0; s < NT; ++s) acc[i][s] = acc_t{0, 0, 0, 0};

  // int8: the tile's bytes from kb on to the stage's end are cleared in LDS, by
  // the workgroup, before the last stage is used (whatever B holds there then
  // meets zeros; 16-bit operands come padded)
  auto clear_last = [&](int buf) {
    if (KIND != kTypeI8 || kb % kStageBytes == 0) return;
    const int at = kb % kStageBytes;
    const int r = threadIdx.x;  // a row per thread
    for (int c = at / 16; c < 16; ++c) {
      u32x4_t* p = &xa[buf][16 * r + (c ^ (r & 15))];
      *p = clear_tail(*p, 16 * c, at);
    }
    __syncthreads();
  };

  u32x4_t b0[NT][STEPS], b1[NT][STEPS];
#pragma unroll
  for (int j = 0; j < 16; ++j)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        at_stage(ar_[j / 4], 0), (__attribute__((address_space(3))) void*)(&xa[0][(16 * wave + j) * 64]), 16,
        xo[j % 4], 0, 0, 0);
#pragma unroll
  for (int j = 0; j < NT * STEPS; ++j)
    b0[j / STEPS][j % STEPS] = buf_load128(at_stage(br_[j / STEPS], 0), bo + 64 * (j % STEPS));
#pragma unroll
  for (int j = 0; j < NT * STEPS; ++j) asm volatile("" ::"v"(b0[j / STEPS][j % STEPS]));
  __builtin_amdgcn_s_waitcnt(kWaitVm0Big);
  __syncthreads();
  if (nst == 1) clear_last(0);

  auto stage = [&](int st, const u32x4_t (&b)[NT][STEPS], u32x4_t (&bn)[NT][STEPS]) {
    const int buf = st & 1;
    const int sn = min(st + 1, nst - 1);  // the last stage is read once more, unused
    buf_t ab[4], bb[NT];
#pragma unroll
    for (int i = 0; i < 4; ++i) ab[i] = at_stage(ar_[i], sn);
#pragma unroll
    for (int s = 0; s < NT; ++s) bb[s] = at_stage(br_[s], sn);
    // opaque here, so that the sums with constants below become the loads'
    // immediate offsets and not registers of their own across the K loop
    int bv = bo;
    asm volatile("" : "+v"(bv));
    const u32x4_t* xs = &xa[buf][0];
    auto frag = [&](int t) {  // operand of row tile t % MT, k step t / MT
      return xs[256 * (t % MT) + 16 * l16 + ((4 * (t / MT) + quad) ^ l16)];
    };
    // While the MFMAs of row tile t run: the operand AHEAD tiles later is read
    // from LDS and one or two loads of the next stage go out
    constexpr int AHEAD = 3, LOADS = 16 + NT * STEPS, SPAN = STEPS * MT / 2;
    u32x4_t ar[AHEAD];
#pragma unroll
    for (int q = 0; q < AHEAD; ++q) ar[q] = frag(q);
#pragma unroll
    for (int t = 0; t < STEPS * MT; ++t) {
      const u32x4_t a = ar[0];
      u32x4_t an = a;
      if (t + AHEAD < STEPS * MT) an = frag(t + AHEAD);
#pragma unroll
      for (int s = 0; s < NT; ++s) mfma_pinned<KIND>(acc[t % MT][s], a, b[s][t / MT]);
#pragma unroll
      for (int j = 0; j < LOADS; ++j)
        if (j * SPAN / LOADS == t) {
          if (j < 16) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                ab[j / 4], (__attribute__((address_space(3))) void*)(&xa[buf ^ 1][(16 * wave + j) * 64]),
                16, xo[j % 4], 0, 0, 0);
          } else {
            const int s = (j - 16) / STEPS, k = (j - 16) % STEPS;
            bn[s][k] = buf_load128(bb[s], bv + 64 * k);
          }
        }
#pragma unroll
      for (int q = 0; q + 1 < AHEAD; ++q) ar[q] = ar[q + 1];
      ar[AHEAD - 1] = an;
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_waitcnt(kWaitVm0Big);
    __syncthreads();
    if (st + 2 == nst) clear_last(buf ^ 1);
  };
  int st = 0;
  for (; st + 1 < nst; st += 2) {
    stage(st, b0, b1);
    stage(st + 1, b1, b0);
  }
  if (st < nst) stage(st, b0, b1);
  // the accumulators were last written by MFMAs that the compiler does not see
  // as such: give them their latency, then pass each through an empty asm
  // ordered after that, so that no read of one moves above it
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int s = 0; s < NT; ++s) asm volatile("" : "+a"(acc[i][s]));
  __builtin_amdgcn_sched_barrier(0);

  uint32_t* t0 = reinterpret_cast<uint32_t*>(lds) + wave * EPI_WORDS;
  Epilogue<KIND, EPI, NT, DT> epi;
  epi.init(g, n0, lane);
  epi.fetch(g, m0);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < MT / 2; ++i)
      put_tile<KIND, NT>(acc[h * MT / 2 + i], t0 + i * epi_words(NT), lane);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll 1
    for (int i = 0; i < MT / 2; ++i) {
      const int r = 16 * (h * MT / 2 + i);
      epi.tile(g, t0 + i * epi_words(NT), sa + r, t0 + (MT / 2) * epi_words(NT), m0 + r, m0 + r + 16);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

template <int KIND, int EPI, int NT, int DT>
__global__ __launch_bounds__(256, 1) void large_kernel(TileArgs g, int n_tiles, int m_tiles) {
  __shared__ u32x4_t lds[LargeLds<EPI, NT>::WORDS16];
  // one array for everything: with a second one in LDS the compiler waits for
  // all memory before LDS reads in the K loop (4096 x 16384 x 8192: 910 us, 470 with one)
  large_body<KIND, EPI, NT, DT>(g, n_tiles, m_tiles, lds);
}

// ---------------------------------------------------------------- host side
template <int KIND, int EPI, int DT>
static hipError_t launch(const TileArgs& t, hipStream_t s) {
  constexpr int NT = 4;
  constexpr int cpg = 4 * (EPI == EPI_GATED || EPI == EPI_GRAD ? 8 : 16) * NT;
  const int64_t cols = EPI == EPI_GRAD ? t.Np : t.N;
  const int64_t rows = EPI == EPI_GRAD && t.dt != nullptr ? t.Mp : t.M;
  const int64_t n_tiles = (cols + cpg - 1) / cpg, m_tiles = (rows + 255) / 256;
  if (n_tiles * m_tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
  return launch_kernel(large_kernel<KIND, EPI, NT, DT>, dim3((unsigned)(n_tiles * m_tiles)),
                       dim3(256), s, t, (int)n_tiles, (int)m_tiles);
}

hipError_t launch_large_scale(const TileArgs& t, hipStream_t s) {
  return launch<kTypeI8, EPI_SCALE, XF16>(t, s);
}
hipError_t launch_large_gated(const TileArgs& t, hipStream_t s) {
  return launch<kTypeI8, EPI_GATED, XF16>(t, s);
}
hipError_t launch_large_grad(const TileArgs& t, int dtype, hipStream_t s) {
  return dtype == XF16 ? launch<kTypeI8, EPI_GRAD, XF16>(t, s) : launch<kTypeI8, EPI_GRAD, XBF16>(t, s);
}
hipError_t launch_large_plain(const TileArgs& t, int dtype, hipStream_t s) {
  return dtype == XF16 ? launch<XF16, EPI_PLAIN, XF16>(t, s) : launch<XBF16, EPI_PLAIN, XBF16>(t, s);
}

}  // namespace qmm
