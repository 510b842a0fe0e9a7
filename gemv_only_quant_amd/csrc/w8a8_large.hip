// w8a8_large.hip -- C = A B^t on the matrix cores for more rows than a decode batch:
// int8 codes (v_mfma_i32_16x16x64_i8, exact sums) and the 16-bit operands of
// gradients (v_mfma_f32_16x16x32_{f16,bf16}).  Both operands have the contracted
// axis contiguous, and one 16-byte chunk per lane is one operand of either kind of
// MFMA (16 int8 or 8 16-bit values), so one kernel moves bytes and only the
// instruction differs.  Epilogues (w8a8_tile.h):
//   SCALE    y = C sa[m] sb[n]
//   GATED    h = act(g) u for two products g, u of the same left operand
//   GRAD     dg = dh u act'(g), du = dh act(g), left as 16-bit operands of the
//            gradients' products, once row-major and once transposed
//   PLAIN    y = C * (a power of two), 16-bit
//   PARTIAL  fp32 sums of a share of the contraction, added by a second launch
//
// Tiles of 256 x 256 (W = 8), bound by the matrix cores, as described here; 128 x
// 128 (W = 4, two workgroups per CU) where the former are too few.
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

// W: 16 x 16 tiles of a wave in each direction; a workgroup's tile is 32 W rows
// and columns of B
constexpr int kLargeStage = 128;  // contracted bytes per stage
// s_waitcnt vmcnt(n) lgkmcnt(0)
static constexpr int wait_mem(int n) { return (n & 15) | ((n >> 4) << 14) | 0x0070; }

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

// LDS of a workgroup in 16-byte words: NB stages of both operands, and in
// their place later the epilogue's tiles (4 waves of as many words each); then
// the row scales.
template <int EPI, int W, int NB> struct LargeLds {
  static constexpr int G = EPI == EPI_GRAD ? 2 : 4;  // row tiles of a wave in LDS at once
  static constexpr int EPI_WORDS = G * epi_words(W) + (EPI == EPI_GRAD ? epi_t_words(W) : 0);
  static constexpr int OPERAND = 32 * W * kLargeStage / 16;  // one operand of a stage
  static constexpr int STAGES = 2 * NB * OPERAND;
  static constexpr int SCALES = STAGES > EPI_WORDS ? STAGES : EPI_WORDS;
  static constexpr int WORDS16 = SCALES + 32 * W / 4;
};

// (a device function beside its kernel: the host pass drops a kernel whose own
// body has matrix-core registers in inline asm)
template <int KIND, int EPI, int W, int NB, int DT>
__device__ __forceinline__ void large_body(const TileArgs& g, int n_tiles, int m_tiles, int per,
                                           u32x4_t* lds) {
  constexpr bool PAIR = EPI == EPI_GATED || EPI == EPI_GRAD;
  constexpr int MT = W, NT = W, TILE = 32 * W, HALF = 16 * W;
  typedef LargeLds<EPI, W, NB> L;
  constexpr int CPW = PAIR ? 8 * NT : 16 * NT;  // output columns per wave
  constexpr int OPERAND = L::OPERAND, EPI_WORDS = L::EPI_WORDS;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, quad = lane >> 4;
  int mt, nt;
  // EPI_PARTIAL: column tiles of every share of K in turn, `per` stages each
  tile_of((int)blockIdx.x, n_tiles, m_tiles, &mt, &nt);
  int k0 = 0, part = 0;
  if constexpr (EPI == EPI_PARTIAL) {
    const int each = (g.N + TILE - 1) / TILE;
    part = nt / each;
    k0 = part * per;
    nt %= each;
  }
  const int m0 = mt * TILE, nw = nt * 2 * CPW;  // the workgroup's first row and column
  const int wm = wave >> 1, wn = wave & 1;
  const int kb = g.kb;
  const int all = (kb + kLargeStage - 1) / kLargeStage;
  const int nst = EPI == EPI_PARTIAL ? min(per, all - k0) : all;
  k0 *= kLargeStage;
  const int kb16 = (kb + 15) & ~15;
  const int lda = (int)g.lda, ldb = (int)g.ldb;

  // One buffer per 16 rows of either operand that this wave moves (8 W of each):
  // the lanes' offsets are then the same few registers for all of them.
  auto rows_of = [&](const void* p, int64_t ld, int first, int limit) {
    const int n = min(16, limit - first);
    return make_buf(static_cast<const char*>(p) + (int64_t)(n > 0 ? first : 0) * ld,
                    n > 0 ? (uint32_t)((n - 1) * (int)ld + kb16) : 0u);
  };
  constexpr int PIECES = W / 2;
  buf_t ra[PIECES], rb[PIECES];
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    ra[i] = rows_of(g.a, g.lda, m0 + 16 * (PIECES * wave + i), g.M);
    // strip PIECES wave + i: NT for each half of the workgroup's columns; of a
    // pair of products, half of them the first's and half the second's
    const int s = PIECES * wave + i, half = s / NT, k = s % NT;
    rb[i] = PAIR ? rows_of(g.b[k / (NT / 2)], g.ldb, nw + half * CPW + 16 * (k % (NT / 2)), g.N)
                 : rows_of(g.b[0], g.ldb, nw + half * CPW + 16 * k, g.N);
  }

  // Load unit u (1 KiB) is rows 8 u .. + 7: lane p's 16 bytes land at slot 64 u +
  // p, so it fetches chunk (p % 8) ^ (r / 2 % 8) of row r = 8 u + p / 8.
  int ao[2], bo[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int chunk = 16 * ((lane & 7) ^ ((4 * c + (lane >> 4)) & 7));
    ao[c] = (8 * c + (lane >> 3)) * lda + chunk + k0;
    bo[c] = (8 * c + (lane >> 3)) * ldb + chunk + k0;
  }
  // load j (W of A, then W of B) of this wave's share of stage st, whose lanes' offsets
  // stand in ao and bo; next_stage moves them on, past the last stage not at all
  // (it is read again, unused)
  auto load = [&](int j, int st) {
    u32x4_t* to = lds + (2 * (st % NB) + j / W) * OPERAND + (W * wave + j % W) * 64;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(j < W ? ra[j / 2] : rb[j % W / 2],
                                             (__attribute__((address_space(3))) void*)to, 16,
                                             j < W ? ao[j % 2] : bo[j % 2], 0, 0, 0);
  };
  auto next_stage = [&](int st) {
    const int d = st < nst ? kLargeStage : 0;
#pragma unroll
    for (int c = 0; c < 2; ++c) ao[c] += d, bo[c] += d;
  };
  // operand i (W of A, then W of B) of k step k of stage st
  const int swz = (l16 >> 1) & 7;
  const int oa = (HALF * wm + l16) * 8, ob = OPERAND + (HALF * wn + l16) * 8;
  auto frag = [&](int i, int k, int st) {
    return lds[2 * (st % NB) * OPERAND + (i < W ? oa + 128 * i : ob + 128 * (i - W)) + ((4 * k + quad) ^ swz)];
  };

  float* sa = reinterpret_cast<float*>(lds + L::SCALES);
  row_scales<EPI>(g, sa, m0, TILE);

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
    for (int c = r < TILE ? at / 16 : 8; c < 8; ++c) {
      u32x4_t* p = lds + 2 * (st % NB) * OPERAND + 8 * r + (c ^ ((r >> 1) & 7));
      *p = clear_tail(*p, 16 * c, at);
    }
    __syncthreads();
  };

  u32x4_t f[2][2 * W];  // operands of the two k steps
#pragma unroll
  for (int q = 0; q < NB; ++q) {
    if (q > 0) next_stage(q);
#pragma unroll
    for (int j = 0; j < 2 * W; ++j) load(j, q);
  }
  __builtin_amdgcn_s_waitcnt(wait_mem((NB - 1) * 2 * W));
  __syncthreads();
  if (nst == 1) clear_last(0);
#pragma unroll
  for (int i = 0; i < 2 * W; ++i) f[0][i] = frag(i, 0, 0);

#pragma unroll 1
  for (int st = 0; st < nst; ++st) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      // groups of 4 MFMAs; the next k step's operands are read in the first half
      // of them, in the order of their first use, and in the second k step the
      // loads go out
      constexpr int GROUPS = W * W / 4, READS = 2 * W, PER = 2 * READS / GROUPS;
#pragma unroll
      for (int t = 0; t < GROUPS; ++t) {
        if (t < GROUPS / 2) {
#pragma unroll
          for (int h = 0; h < PER; ++h) {
            const int q = PER * t + h, i = q == 0 ? 0 : (q <= W ? W + q - 1 : q - W);
            f[k ^ 1][i] = frag(i, k ^ 1, st + k);
          }
        }
        if (k == 1) {
#pragma unroll
          for (int j = t * READS / GROUPS; j < (t + 1) * READS / GROUPS; ++j) load(j, st + NB);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int i = t * 4 / W, c = t * 4 % W + s;
          mfma_pinned<KIND>(acc[i][c], f[k][i], f[k][W + c]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (k == 0) {
        __builtin_amdgcn_s_waitcnt(wait_mem((NB - 2) * 2 * W));
        __syncthreads();
        if (st + 2 == nst) clear_last(st + 1);
        next_stage(st + NB);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  __builtin_amdgcn_s_waitcnt(wait_mem(0));
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
  const int mw = m0 + HALF * wm, rw = HALF * wm;  // the wave's first row; in the tile
  TileArgs ge = g;
  if constexpr (EPI == EPI_PARTIAL) ge.y = static_cast<float*>(g.y) + part * ((int64_t)g.M * g.ldy);
  Epilogue<KIND, EPI, NT, DT> epi;
  epi.init(ge, nw + wn * CPW, lane);
  epi.fetch(ge, mw);
  constexpr int G = L::G;
#pragma unroll
  for (int h = 0; h < MT / G; ++h) {
#pragma unroll
    for (int i = 0; i < G; ++i) put_tile<KIND, NT>(acc[h * G + i], t0 + i * epi_words(NT), lane);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll 1
    for (int i = 0; i < G; ++i) {
      const int r = 16 * (h * G + i);
      epi.tile(ge, t0 + i * epi_words(NT), sa + rw + r, t0 + G * epi_words(NT), mw + r, mw + r + 16);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

template <int KIND, int EPI, int W, int NB, int DT>
__global__ __launch_bounds__(256, W == 4 && NB == 2 ? 2 : 1) void large_kernel(TileArgs g, int n_tiles,
                                                                    int m_tiles, int per) {
  // one array for everything: with a second one in LDS the compiler waits for
  // all memory before LDS reads in the K loop
  __shared__ u32x4_t lds[LargeLds<EPI, W, NB>::WORDS16];
  large_body<KIND, EPI, W, NB, DT>(g, n_tiles, m_tiles, per, lds);
}

// ---------------------------------------------------------------- host side
// Tiles of a product with tiles of 32 W, in n (pairs of products: half as many
// columns) and m.
static int64_t tiles_of(int64_t m, int64_t n, bool pair, int w) {
  const int64_t rows = 32 * w, cols = pair ? 16 * w : 32 * w;
  return ((m + rows - 1) / rows) * ((n + cols - 1) / cols);
}

// Whether 256 x 256 tiles serve a product better than 128 x 128 ones, in units
// of the time of a round of the former (K = 4096: 54 us).  Of the latter a CU
// runs two at once (42 us together), or where there are at most 256, one with
// twice the stages in flight (24 us).  So 1024 x 4096 x 4096 takes 25 us and not
// 54, 512 x 4096 x 11008 42 and not 56, 1024 x 4096 x 11008 56 and not 73.
static bool large_tiles(int64_t m, int64_t n, bool pair) {
  const int64_t t8 = tiles_of(m, n, pair, 8), t4 = tiles_of(m, n, pair, 4);
  const double small = t4 <= 256 ? 0.45 : 0.77 * (double)((t4 + 511) / 512);
  return (double)((t8 + 255) / 256) <= small;
}

template <int KIND, int EPI, int W, int NB, int DT>
static hipError_t launch_w(const TileArgs& t, int64_t m, int64_t n, hipStream_t s) {
  constexpr int rows = 32 * W, cols = EPI == EPI_GATED || EPI == EPI_GRAD ? 16 * W : 32 * W;
  int64_t n_tiles = (n + cols - 1) / cols;
  const int64_t m_tiles = (m + rows - 1) / rows;
  int per = 0;
  if constexpr (EPI == EPI_PARTIAL) {
    per = (t.kb / kLargeStage + t.splits - 1) / t.splits;
    n_tiles *= t.splits;
  }
  if (n_tiles * m_tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
  return launch_kernel(large_kernel<KIND, EPI, W, NB, DT>, dim3((unsigned)(n_tiles * m_tiles)), dim3(256),
                       s, t, (int)n_tiles, (int)m_tiles, per);
}

template <int KIND, int EPI, int DT>
static hipError_t launch(const TileArgs& t, hipStream_t s) {
  // the gradient epilogue also writes the padding of its operands
  const int64_t n = EPI == EPI_GRAD ? t.Np : t.N;
  const int64_t m = EPI == EPI_GRAD && t.dt != nullptr ? t.Mp : t.M;
  if constexpr (EPI == EPI_PARTIAL) return launch_w<KIND, EPI, 8, 2, DT>(t, m, n, s);
  constexpr bool pair = EPI == EPI_GATED || EPI == EPI_GRAD;
  if (large_tiles(m, n, pair)) return launch_w<KIND, EPI, 8, 2, DT>(t, m, n, s);
  return tiles_of(m, n, pair, 4) <= 256 ? launch_w<KIND, EPI, 4, 4, DT>(t, m, n, s)
                                        : launch_w<KIND, EPI, 4, 2, DT>(t, m, n, s);
}

hipError_t launch_tile_scale(const TileArgs& t, hipStream_t s) {
  return launch<kTypeI8, EPI_SCALE, XF16>(t, s);
}
hipError_t launch_tile_gated(const TileArgs& t, hipStream_t s) {
  return launch<kTypeI8, EPI_GATED, XF16>(t, s);
}
hipError_t launch_tile_grad(const TileArgs& t, int dtype, hipStream_t s) {
  return dtype == XF16 ? launch<kTypeI8, EPI_GRAD, XF16>(t, s) : launch<kTypeI8, EPI_GRAD, XBF16>(t, s);
}

// y = (sum of the partial products) *scal, rounded once; 4 columns per thread.
template <int DT>
__global__ __launch_bounds__(256) void sum_partials_kernel(TileArgs t, int blocks_per_row) {
  typedef typename Half16<DT>::type T;
  const int m = (int)(blockIdx.x / (unsigned)blocks_per_row);
  const int n = ((int)(blockIdx.x % (unsigned)blocks_per_row) * 256 + (int)threadIdx.x) * 4;
  const bool second = m >= t.M2;
  const int mo = second ? m - t.M2 : m;
  if (n >= t.N || mo >= t.Mv) return;
  const int64_t ld = round_up(t.N, 4), at = (int64_t)m * ld + n;
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < t.splits; ++s)
    v += *reinterpret_cast<const f32x4_t*>(t.part + s * (int64_t)t.M * ld + at);
  const float k = *t.scal;
  T* y = static_cast<T*>(second ? t.y2 : t.y) + (int64_t)mo * t.ldy + n;
  const float o[4] = {v[0] * k, v[1] * k, v[2] * k, v[3] * k};
  store4(y, o, min(4, t.N - n), vec4_ok(second ? t.y2 : t.y, t.ldy, 2));
}

int plain_splits(int64_t M, int64_t N, int64_t kb) {
  const int64_t tiles = tiles_of(M, N, false, 8);
  // shares of K that fill the CUs, none of them under 16 stages (1024 values)
  int64_t s = 256 / tiles;
  s = s < kb / kLargeStage / 16 ? s : kb / kLargeStage / 16;
  if (s < 2) return 1;
  // the same number of stages in all but the last, which is not empty
  const int64_t per = (kb / kLargeStage + s - 1) / s;
  return (int)((kb / kLargeStage + per - 1) / per);
}

hipError_t launch_tile_plain(const TileArgs& t, int dtype, hipStream_t s) {
  if (t.splits > 1) {
    TileArgs p = t;
    p.y = t.part;
    p.ldy = round_up(t.N, 4);
    p.y_dtype = YF32;
    hipError_t e = dtype == XF16 ? launch<XF16, EPI_PARTIAL, XF16>(p, s) : launch<XBF16, EPI_PARTIAL, XBF16>(p, s);
    if (e != hipSuccess) return e;
    const int bpr = (t.N + 1023) / 1024;
    const dim3 grid((unsigned)((int64_t)t.M * bpr));
    return dtype == XF16 ? launch_kernel(sum_partials_kernel<XF16>, grid, dim3(256), s, t, bpr)
                         : launch_kernel(sum_partials_kernel<XBF16>, grid, dim3(256), s, t, bpr);
  }
  return dtype == XF16 ? launch<XF16, EPI_PLAIN, XF16>(t, s) : launch<XBF16, EPI_PLAIN, XBF16>(t, s);
}

}  // namespace qmm
