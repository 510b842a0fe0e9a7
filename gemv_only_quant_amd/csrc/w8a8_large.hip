// w8a8_large.hip -- the products of w8a8_tile.hip for many rows: 256 x 256
// tiles, bound by the matrix cores.
//
//  * one workgroup per CU, 4 waves as 2 x 2; a wave owns 128 rows x 128 columns
//    = 8 x 8 MFMA tiles, 256 accumulators per lane pinned to the matrix-core
//    (AGPR) registers;
//  * a stage is 128 contracted bytes (128 int8 or 64 16-bit values), two MFMA k
//    steps.  Both operands' tiles of a stage, 32 KiB each, are shared through
//    double-buffered LDS, filled by buffer loads straight to LDS: whole 128-byte
//    lines, 8 lanes each, 8 rows per load.  Read from LDS they are conflict-free
//    ds_read_b128: chunk c of row r lies at slot 8 r + (c ^ (r / 2 % 8));
//  * 16 operands (8 of A, 8 of B) feed 64 MFMAs, and are read while the 64 of the
//    k step before run.  So when a stage's second k step begins, all of its
//    operands are in registers, its buffer is free, and one barrier there does
//    everything: the next stage's loads have arrived, the one after may go out.
//    Neither loads nor LDS reads nor the barrier leave the matrix cores idle.
// (B from memory straight into operands, 16 rows x 64 bytes per load, was 10%
// slower: neighbouring lanes then lie in different rows, and the address units take
// the 64 lanes one by one; 256 x 256 with the waves side by side and half the
// tile, two workgroups per CU, 24%.)
// Every address is in the offset that the buffer's range is checked against:
// rows past M and columns past N read zeros.
#include "w8a8_tile.h"

namespace qmm {

constexpr int kLargeMT = 8, kLargeNT = 8;  // 16 x 16 tiles of a wave
constexpr int kLargeTile = 256;            // rows and columns of B of a workgroup
constexpr int kLargeStage = 128;           // contracted bytes per stage
constexpr int kLargeEpiTiles = 4;          // row tiles of a wave in the epilogue's LDS at once
static constexpr int kWaitMem = 0x0070;    // s_waitcnt vmcnt(0) lgkmcnt(0)

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

// LDS of a workgroup in 16-byte words: two stages of both operands, and in
// their place later the epilogue's tiles (4 waves of as many words each); then
// the row scales.
template <int EPI> struct LargeLds {
  static constexpr int EPI_WORDS =
      kLargeEpiTiles * epi_words(kLargeNT) + (EPI == EPI_GRAD ? epi_t_words(kLargeNT) : 0);
  static constexpr int OPERAND = kLargeTile * kLargeStage / 16;  // one operand of a stage
  static constexpr int STAGES = 4 * OPERAND;
  static constexpr int SCALES = STAGES > EPI_WORDS ? STAGES : EPI_WORDS;
  static constexpr int WORDS16 = SCALES + kLargeTile / 4;
};

// (a device function beside its kernel: the host pass drops a kernel whose own
// body has matrix-core registers in inline asm)
template <int KIND, int EPI, int DT>
__device__ __forceinline__ void large_body(const TileArgs& g, int n_tiles, int m_tiles,
                                           u32x4_t* lds) {
  constexpr bool PAIR = EPI == EPI_GATED || EPI == EPI_GRAD;
  constexpr int MT = kLargeMT, NT = kLargeNT;
  constexpr int CPW = PAIR ? 8 * NT : 16 * NT;  // output columns per wave
  constexpr int OPERAND = LargeLds<EPI>::OPERAND, EPI_WORDS = LargeLds<EPI>::EPI_WORDS;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, quad = lane >> 4;
  int mt, nt;
  tile_of((int)blockIdx.x, n_tiles, m_tiles, &mt, &nt);
  const int m0 = mt * kLargeTile, nw = nt * 2 * CPW;  // the workgroup's first row and column
  const int wm = wave >> 1, wn = wave & 1;
  const int kb = g.kb, nst = (kb + kLargeStage - 1) / kLargeStage;
  const int kb16 = (kb + 15) & ~15;
  const int lda = (int)g.lda, ldb = (int)g.ldb;

  // One buffer per 16 rows of either operand that this wave moves (64 of each),
  // from a stage's first byte to the end of the last row: the lanes' offsets are
  // then the same few registers for all of them.
  struct Rows {
    const char* base;
    int range;  // bytes, 0 where no row exists
  };
  auto rows_of = [&](const void* p, int64_t ld, int first, int limit) {
    const int n = min(16, limit - first);
    Rows r;
    r.base = static_cast<const char*>(p) + (int64_t)(n > 0 ? first : 0) * ld;
    r.range = n > 0 ? (int)((n - 1) * ld) + kb16 : 0;
    return r;
  };
  auto at_stage = [&](const Rows& r, int st) {
    return make_buf(r.base + st * kLargeStage, r.range > 0 ? (uint32_t)(r.range - st * kLargeStage) : 0u);
  };
  Rows ra[4], rb[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    ra[i] = rows_of(g.a, g.lda, m0 + 64 * wave + 16 * i, g.M);
    // strip 4 wave + i of the 16: NT for each half of the workgroup's columns; of a
    // pair of products, half of them the first's and half the second's
    const int s = 4 * wave + i, half = s / NT, k = s % NT;
    rb[i] = PAIR ? rows_of(g.b[k / (NT / 2)], g.ldb, nw + half * CPW + 16 * (k % (NT / 2)), g.N)
                 : rows_of(g.b[0], g.ldb, nw + half * CPW + 16 * k, g.N);
  }

  // Load unit u (1 KiB) is rows 8 u .. + 7: lane p's 16 bytes land at slot 64 u +
  // p, so it fetches chunk (p % 8) ^ (r / 2 % 8) of row r = 8 u + p / 8.
  int ao[2], bo[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int chunk = 16 * ((lane & 7) ^ ((4 * c + (lane >> 4)) & 7));
    ao[c] = (8 * c + (lane >> 3)) * lda + chunk;
    bo[c] = (8 * c + (lane >> 3)) * ldb + chunk;
  }
  // load j (0 .. 15) of this wave's share of stage st
  auto load = [&](int j, int st) {
    u32x4_t* to = lds + (2 * (st & 1) + j / 8) * OPERAND + (8 * wave + j % 8) * 64;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        at_stage(j < 8 ? ra[j / 2] : rb[j % 8 / 2], min(st, nst - 1)),  // past the end: unused
        (__attribute__((address_space(3))) void*)to, 16, j < 8 ? ao[j % 2] : bo[j % 2], 0, 0, 0);
  };
  // operand i (0 .. 7 of A, 8 .. 15 of B) of k step k of stage st
  const int swz = (l16 >> 1) & 7;
  const int oa = (128 * wm + l16) * 8, ob = OPERAND + (128 * wn + l16) * 8;
  auto frag = [&](int i, int k, int st) {
    return lds[2 * (st & 1) * OPERAND + (i < 8 ? oa + 128 * i : ob + 128 * (i - 8)) + ((4 * k + quad) ^ swz)];
  };

  float* sa = reinterpret_cast<float*>(lds + LargeLds<EPI>::SCALES);
  row_scales<EPI>(g, sa, m0, kLargeTile);

  typedef typename Acc<KIND>::type acc_t;
  acc_t acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int s = 0; s < NT; ++s) acc[i][s] = acc_t{0, 0, 0, 0};

  // int8: the bytes of A from kb on to the last stage's end are cleared in LDS,
  // by the workgroup, before that stage is read (whatever B holds there then
  // meets zeros; 16-bit operands come padded)
  auto clear_last = [&](int st) {
    if (KIND != kTypeI8 || kb % kLargeStage == 0) return;
    const int at = kb % kLargeStage, r = threadIdx.x;  // a row per thread
    for (int c = at / 16; c < 8; ++c) {
      u32x4_t* p = lds + 2 * (st & 1) * OPERAND + 8 * r + (c ^ ((r >> 1) & 7));
      *p = clear_tail(*p, 16 * c, at);
    }
    __syncthreads();
  };

  u32x4_t f[2][16];  // operands of the two k steps
#pragma unroll
  for (int j = 0; j < 16; ++j) load(j, 0);
  __builtin_amdgcn_s_waitcnt(kWaitMem);
  __syncthreads();
  if (nst == 1) clear_last(0);
#pragma unroll
  for (int j = 0; j < 16; ++j) load(j, 1);
#pragma unroll
  for (int i = 0; i < 16; ++i) f[0][i] = frag(i, 0, 0);

#pragma unroll 1
  for (int st = 0; st < nst; ++st) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      // 16 groups of 4 MFMAs; the next k step's operands are read in the first 8,
      // two with each, and in the second k step the loads go out
#pragma unroll
      for (int t = 0; t < 16; ++t) {
        if (t < 8) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // in the order of their first use: B's first half with A's first
            const int q = 2 * t + h, i = q < 5 ? (q == 0 ? 0 : 7 + q) : (q < 9 ? 7 + q : q - 8);
            f[k ^ 1][i] = frag(i, k ^ 1, st + k);
          }
        }
        if (k == 1) load(t, st + 2);
#pragma unroll
        for (int s = 0; s < 4; ++s)
          mfma_pinned<KIND>(acc[t / 2][4 * (t % 2) + s], f[k][t / 2], f[k][8 + 4 * (t % 2) + s]);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (k == 0) {
        __builtin_amdgcn_s_waitcnt(kWaitMem);
        __syncthreads();
        if (st + 2 == nst) clear_last(st + 1);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  __builtin_amdgcn_s_waitcnt(kWaitMem);
  __syncthreads();  // every wave has left the stages: their LDS becomes the epilogue's
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
  const int mw = m0 + 128 * wm, rw = 128 * wm;  // the wave's first row; in the tile
  Epilogue<KIND, EPI, NT, DT> epi;
  epi.init(g, nw + wn * CPW, lane);
  epi.fetch(g, mw);
  constexpr int G = kLargeEpiTiles;
#pragma unroll
  for (int h = 0; h < MT / G; ++h) {
#pragma unroll
    for (int i = 0; i < G; ++i) put_tile<KIND, NT>(acc[h * G + i], t0 + i * epi_words(NT), lane);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll 1
    for (int i = 0; i < G; ++i) {
      const int r = 16 * (h * G + i);
      epi.tile(g, t0 + i * epi_words(NT), sa + rw + r, t0 + G * epi_words(NT), mw + r, mw + r + 16);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

template <int KIND, int EPI, int DT>
__global__ __launch_bounds__(256, 1) void large_kernel(TileArgs g, int n_tiles, int m_tiles) {
  // one array for everything: with a second one in LDS the compiler waits for
  // all memory before LDS reads in the K loop
  __shared__ u32x4_t lds[LargeLds<EPI>::WORDS16];
  large_body<KIND, EPI, DT>(g, n_tiles, m_tiles, lds);
}

// ---------------------------------------------------------------- host side
template <int KIND, int EPI, int DT>
static hipError_t launch(const TileArgs& t, hipStream_t s) {
  constexpr int cols = EPI == EPI_GATED || EPI == EPI_GRAD ? kLargeTile / 2 : kLargeTile;
  const int64_t n = EPI == EPI_GRAD ? t.Np : t.N;
  const int64_t m = EPI == EPI_GRAD && t.dt != nullptr ? t.Mp : t.M;
  const int64_t n_tiles = (n + cols - 1) / cols, m_tiles = (m + kLargeTile - 1) / kLargeTile;
  if (n_tiles * m_tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
  return launch_kernel(large_kernel<KIND, EPI, DT>, dim3((unsigned)(n_tiles * m_tiles)), dim3(256), s,
                       t, (int)n_tiles, (int)m_tiles);
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
