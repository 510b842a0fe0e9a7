// w8a8_large.hip -- products on the matrix cores for more rows than a decode batch:
// C = A B^t of int8 codes (v_mfma_i32_16x16x64_i8, exact sums), both with the
// contracted axis contiguous, and the gradients' C = A B of 16-bit values by int8
// codes (v_mfma_f32_16x16x32_{f16,bf16}), the contracted axis the codes' rows.
// Epilogues (w8a8_tile.h):
//   SCALE    y = C sa[m] sb[n]
//   GATED    h = act(g) u for two products g, u of the same left operand
//   GRAD     dg = dh u act'(g), du = dh act(g), left as 16-bit operands of the
//            gradients' products, once row-major and once transposed
//   PLAIN    y = C (fp16: times a power of two for each row), 16-bit
//   PARTIAL  fp32 sums of a share of the contraction, added by a second launch
//
// Tiles of 256 x 256 (W = 8), bound by the matrix cores (2.7e15 operations/s of int8
// over many rounds, at the 1.8 GHz that the power limit leaves), as described here;
// 128 x 128 (W = 4, two workgroups per CU) where the former are too few.
//
//  * one workgroup per CU, 4 waves as 2 x 2; a wave owns 128 rows x 128 columns
//    = 8 x 8 MFMA tiles, 256 accumulators per lane pinned to the matrix-core
//    (AGPR) registers;
//  * a stage is 128 contracted bytes of A (128 int8 or 64 16-bit values), two MFMA
//    k steps.  Both operands' tiles of a stage, 32 KiB each, are shared through
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
//  * 16-bit: B's stage is 64 rows of 256 codes, 16 KiB, transposed by LDS reads of 8
//    x 8 bytes, and made 16-bit values between the MFMAs.  The waves lie side by
//    side, 256 rows x 64 columns, so that each code is converted once and not
//    twice (1.0e15 operations/s at 4096 x 22016 x 4096, the library's product of
//    16-bit values 1.56e15).
// Every address is in the offset that the buffer's range is checked against:
// rows past M and columns past N read zeros (codes of columns past N: anything, for
// outputs that are not stored).
#include "w8a8_tile.h"

namespace qmm {

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

// 8 codes of a column as exact 16-bit values, pairs in order.
template <int KIND> __device__ __forceinline__ u32x4_t code_operand(u32x2_t q) {
  u32x4_t o;
  if constexpr (KIND == XF16) {
    // u = q + 128 under the fp16 exponent of 1024 gives 1024 + u; less 1152 it is q
    const half2_t off = {(_Float16)-1152.0f, (_Float16)-1152.0f};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t u = q[j / 2] ^ 0x80808080u;
      const uint32_t p = __builtin_amdgcn_perm(0x64646464u, u, j % 2 ? 0x04030402u : 0x04010400u);
      o[j] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, p) + off);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w = q[j / 2];
      const int sh = 16 * (j % 2);
      const bf16x2_t p = {(__bf16)(float)(int8_t)(w >> sh), (__bf16)(float)(int8_t)(w >> (sh + 8))};
      o[j] = __builtin_bit_cast(uint32_t, p);
    }
  }
  return o;
}

// A buffer descriptor (make_buf's) as the four words it consists of, and a load
// of 16 bytes per lane through it straight to LDS, the wave's 1 KiB from `to` on.
// Written out for the kernels that read LDS transposed: before such a read the
// compiler waits for every load to LDS that it knows to be in flight, while the
// kernel's own waits and barriers say when they have arrived.  (It has no register
// to write.)
__device__ __forceinline__ u32x4_t buf_words(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return u32x4_t{(uint32_t)a, (uint32_t)(a >> 32) & 0xFFFFu, bytes, 0x00020000u};
}
__device__ __forceinline__ void load_to_lds(const u32x4_t& buf, int off, u32x4_t* to) {
  const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)to;
  // the wait states cover a descriptor word that a vector instruction has just
  // written (a spilled one's reload), for which a load has to stand back 5
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(at),
               "v"(off), "s"(buf)
               : "memory", "m0");
}

template <bool WORDS> struct LdsLoad {
  typedef u32x4_t buf;
  static __device__ __forceinline__ buf make(const void* p, uint32_t n) { return buf_words(p, n); }
  static __device__ __forceinline__ void go(const buf& b, int off, u32x4_t* to) { load_to_lds(b, off, to); }
};
template <> struct LdsLoad<false> {
  typedef buf_t buf;
  static __device__ __forceinline__ buf make(const void* p, uint32_t n) { return make_buf(p, n); }
  static __device__ __forceinline__ void go(const buf& b, int off, u32x4_t* to) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (__attribute__((address_space(3))) void*)to, 16, off, 0, 0, 0);
  }
};

// LDS of a workgroup in 16-byte words: NB stages of both operands, and in
// their place later the epilogue's tiles (4 waves of as many words each); then
// the row scales.
template <int KIND, int EPI, int W, int NB> struct LargeLds {
  static constexpr int MT = KIND == kTypeI8 ? W : 2 * W, NT = KIND == kTypeI8 ? W : W / 2;
  static constexpr int G = EPI == EPI_GRAD ? 2 : 4;  // row tiles of a wave in LDS at once
  static constexpr int EPI_WORDS = G * epi_words(NT) + (EPI == EPI_GRAD ? epi_t_words(NT) : 0);
  static constexpr int A = 32 * W * kStageBytes / 16;      // A of a stage
  static constexpr int B = KIND == kTypeI8 ? A : A / 2;    // B: as A, or codes
  static constexpr int STAGES = NB * (A + B);
  static constexpr int SCALES = STAGES > EPI_WORDS ? STAGES : EPI_WORDS;
  static constexpr int WORDS16 = SCALES + 32 * W / 4;
};

// W: a workgroup's tile is 32 W rows and columns of B, a wave's W x W tiles of 16 x 16
// (codes: 2 W x W / 2); NB stages are in flight.
// (a device function beside its kernel: the host pass drops a kernel whose own
// body has matrix-core registers in inline asm)
template <int KIND, int EPI, int W, int NB, int DT>
__device__ __forceinline__ void large_body(const TileArgs& g, int n_tiles, int m_tiles, int per,
                                           u32x4_t* lds) {
  constexpr bool PAIR = EPI == EPI_GATED || EPI == EPI_GRAD;
  typedef LargeLds<KIND, EPI, W, NB> L;
  constexpr int MT = L::MT, NT = L::NT, TILE = 32 * W;
  constexpr bool CODES = KIND != kTypeI8;  // B is int8 codes, the contracted axis its rows
  constexpr int CPW = PAIR ? 8 * NT : 16 * NT;  // output columns per wave
  constexpr int STAGE = L::A + L::B, EPI_WORDS = L::EPI_WORDS;

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
  const int m0 = mt * TILE, nw = nt * (PAIR ? TILE / 2 : TILE);  // the workgroup's first row and column
  // waves as 2 x 2, or side by side where B is codes: each is then converted once
  const int wm = CODES ? 0 : wave >> 1, wn = CODES ? wave : wave & 1;
  const int kb = g.kb;
  const int all = (kb + kStageBytes - 1) / kStageBytes;
  const int nst = EPI == EPI_PARTIAL ? min(per, all - k0) : all;
  k0 *= kStageBytes;
  const int kb16 = (kb + 15) & ~15;
  const int lda = (int)g.lda, ldb = (int)g.ldb;

  // One buffer per 16 rows of either operand that this wave moves (8 W of each):
  // the lanes' offsets are then the same few registers for all of them.
  typedef LdsLoad<CODES> Load;
  auto rows_of = [&](const void* p, int64_t ld, int first, int limit) {
    const int n = min(16, limit - first);
    return Load::make(static_cast<const char*>(p) + (int64_t)(n > 0 ? first : 0) * ld,
                     n > 0 ? (uint32_t)((n - 1) * (int)ld + kb16) : 0u);
  };
  constexpr int PIECES = W / 2;
  typename Load::buf ra[PIECES], rb[PIECES];
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    ra[i] = rows_of(g.a, g.lda, m0 + 16 * (PIECES * wave + i), g.M);
    // strip PIECES wave + i: NT for each half of the workgroup's columns; of a
    // pair of products, half of them the first's and half the second's
    const int s = PIECES * wave + i, half = s / NT, k = s % NT;
    if constexpr (!CODES)
      rb[i] = PAIR ? rows_of(g.b[k / (NT / 2)], g.ldb, nw + half * CPW + 16 * (k % (NT / 2)), g.N)
                   : rows_of(g.b[0], g.ldb, nw + half * CPW + 16 * k, g.N);
  }
  // Codes: this wave moves 16 of a stage's 64 rows, the workgroup's columns of
  // each.  Rows come in parts of g.brows that exist, padded to g.bpad (what is
  // read for the padding meets zeros of A, whatever codes it is); columns past N
  // feed outputs that are not stored.
  auto code_rows = [&](int st) {
    const int j = 64 * st + 16 * wave, part = j >= g.bpad ? 1 : 0, r = j - part * g.bpad;
    const int n = min(16, g.brows - r);
    const int cols = (min(TILE, g.N - nw) + 15) & ~15;
    return buf_words(static_cast<const char*>(g.b[part]) + (int64_t)(n > 0 ? r : 0) * ldb + nw,
                     n > 0 ? (uint32_t)((n - 1) * ldb + cols) : 0u);
  };

  // Load unit u (1 KiB) is rows 8 u .. + 7: lane p's 16 bytes land at slot 64 u +
  // p, so it fetches chunk (p % 8) ^ (r / 2 % 8) of row r = 8 u + p / 8.
  int ao[2], bo[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int chunk = 16 * ((lane & 7) ^ ((4 * c + (lane >> 4)) & 7));
    ao[c] = (8 * c + (lane >> 3)) * lda + chunk + k0;
    bo[c] = (8 * c + (lane >> 3)) * ldb + chunk + k0;
  }
  // Codes in LDS: chunk c (of 2 W) of row r at c ^ code_swz(r); a load unit is 32
  // / W rows.
  constexpr int CH = 2 * W, CODE_UNITS = W / 2;
  auto code_swz = [](int r) { return W == 8 ? r & 15 : (r >> 1) & 7; };
  int co[CODES ? CODE_UNITS : 1];
  if constexpr (CODES) {
#pragma unroll
    for (int u = 0; u < CODE_UNITS; ++u) {
      const int r = 64 / CH * u + lane / CH;  // of the wave's 16
      co[u] = r * ldb + 16 * ((lane % CH) ^ code_swz(r));
    }
  }
  // load j (W of A, then B's) of this wave's share of stage st, whose lanes'
  // offsets stand in ao and bo; next_stage moves them on, past the last stage not
  // at all (it is read again, unused)
  constexpr int LOADS = W + (CODES ? CODE_UNITS : W);
  u32x4_t cb = {0u, 0u, 0u, 0u};
  if constexpr (CODES) cb = code_rows(k0 / kStageBytes);
  auto load = [&](int j, int st) {
    u32x4_t* at = lds + st % NB * STAGE;
    if (j < W) Load::go(ra[j / 2], ao[j % 2], at + (W * wave + j) * 64);
    else if constexpr (CODES) Load::go(cb, co[j - W], at + L::A + (CODE_UNITS * wave + j - W) * 64);
    else Load::go(rb[(j - W) / 2], bo[j % 2], at + L::A + (W * wave + j - W) * 64);
  };
  auto next_stage = [&](int st) {
    const int d = st < nst ? kStageBytes : 0;
#pragma unroll
    for (int c = 0; c < 2; ++c) ao[c] += d, bo[c] += d;
    if constexpr (CODES) cb = code_rows(k0 / kStageBytes + min(st, nst - 1));
  };
  // operand i (MT of A, then NT of B) of k step k of stage st
  const int swz = (l16 >> 1) & 7;
  const int oa = (16 * MT * wm + l16) * 8, ob = L::A + (16 * NT * wn + l16) * 8;
  auto frag = [&](int i, int k, int st) {
    return lds[st % NB * STAGE + (i < MT ? oa + 128 * i : ob + 128 * (i - MT)) + ((4 * k + quad) ^ swz)];
  };
  // Codes of strip c and k step k: 8 rows' bytes of a column per lane.  The LDS
  // transposes 8 x 8 bytes within 16 lanes: lane i of them names 8 columns (i % 2)
  // of row i / 2, lane l receives column l of the 8 rows.
  auto code_frag = [&](int c, int k, int st) {
    const int r = 32 * k + 8 * quad + (l16 >> 1);
    const char* at = reinterpret_cast<const char*>(lds + st % NB * STAGE + L::A) + r * (32 * W) +
                     16 * ((NT * wn + c) ^ code_swz(r)) + 8 * (l16 & 1);
    typedef int i32x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr8_b64_v2i32(
        (__attribute__((address_space(3))) i32x2_t*)at));
  };

  float* sa = reinterpret_cast<float*>(lds + L::SCALES);
  row_scales<EPI, DT>(g, sa, m0, TILE);

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
    if (KIND != kTypeI8 || kb % kStageBytes == 0) return;
    const int at = kb % kStageBytes, r = threadIdx.x;  // a row per thread
    for (int c = r < TILE ? at / 16 : 8; c < 8; ++c) {
      u32x4_t* p = lds + st % NB * STAGE + 8 * r + (c ^ ((r >> 1) & 7));
      *p = clear_tail(*p, 16 * c, at);
    }
    __syncthreads();
  };

  u32x4_t f[2][MT + NT];  // operands of the two k steps
  u32x2_t raw[NT];
#pragma unroll
  for (int q = 0; q < NB; ++q) {
    if (q > 0) next_stage(q);
#pragma unroll
    for (int j = 0; j < LOADS; ++j) load(j, q);
  }
  __builtin_amdgcn_s_waitcnt(wait_mem((NB - 1) * LOADS));
  __syncthreads();
  if (nst == 1) clear_last(0);
#pragma unroll
  for (int i = 0; i < MT + NT; ++i) {
    if (CODES && i >= MT) f[0][i] = code_operand<KIND>(code_frag(i - MT, 0, 0));
    else f[0][i] = frag(i, 0, 0);
  }

#pragma unroll 1
  for (int st = 0; st < nst; ++st) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      // groups of 4 MFMAs; the next k step's operands are read in the first half
      // of them, in the order of their first use (codes in the first quarter,
      // and made operands between the MFMAs of the rest), and in the second k
      // step the loads go out
      constexpr int GROUPS = W * W / 4, PER = 4 * W / GROUPS, Q = GROUPS / 4;
#pragma unroll
      for (int t = 0; t < GROUPS; ++t) {
        if (!CODES && t < GROUPS / 2) {
#pragma unroll
          for (int h = 0; h < PER; ++h) {
            const int q = PER * t + h, i = q == 0 ? 0 : (q <= W ? W + q - 1 : q - W);
            f[k ^ 1][i] = frag(i, k ^ 1, st + k);
          }
        }
        if (CODES && t < Q) {
#pragma unroll
          for (int c = t * NT / Q; c < (t + 1) * NT / Q; ++c) raw[c] = code_frag(c, k ^ 1, st + k);
        }
        if (CODES && t < 2 * Q) {
#pragma unroll
          for (int i = t * MT / (2 * Q); i < (t + 1) * MT / (2 * Q); ++i) f[k ^ 1][i] = frag(i, k ^ 1, st + k);
        }
        if (CODES && t >= Q) {
#pragma unroll
          for (int c = (t - Q) * NT / (3 * Q); c < (t - Q + 1) * NT / (3 * Q); ++c)
            f[k ^ 1][MT + c] = code_operand<KIND>(raw[c]);
        }
        if (k == 1) {
#pragma unroll
          for (int j = t * LOADS / GROUPS; j < (t + 1) * LOADS / GROUPS; ++j) load(j, st + NB);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int i = (4 * t + s) / NT, c = (4 * t + s) % NT;
          mfma_pinned<KIND>(acc[i][c], f[k][i], f[k][MT + c]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (k == 0) {
        __builtin_amdgcn_s_waitcnt(wait_mem((NB - 2) * LOADS));
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
  const int mw = m0 + 16 * MT * wm, rw = 16 * MT * wm;  // the wave's first row; in the tile
  TileArgs ge = g;
  if constexpr (EPI == EPI_PARTIAL) ge.y = static_cast<float*>(g.y) + part * ((int64_t)g.M * g.ldy);
  Epilogue<KIND, EPI, NT, DT> epi;
  epi.init(ge, nw + wn * CPW, lane);
  epi.fetch(ge, mw);
  constexpr int G = L::G;
  // the activation is a constant of the loop over tiles, and not of its body alone: with
  // three of them inside, the fp16 gradient's loop is beyond what the compiler unrolls,
  // and the accumulators go to memory
  auto tiles = [&](auto act) {
#pragma unroll
    for (int h = 0; h < MT / G; ++h) {
#pragma unroll
      for (int i = 0; i < G; ++i) put_tile<KIND, NT>(acc[h * G + i], t0 + i * epi_words(NT), lane);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll 1
      for (int i = 0; i < G; ++i) {
        const int r = 16 * (h * G + i);
        epi.template tile<decltype(act)::value>(ge, t0 + i * epi_words(NT), sa + rw + r, t0 + G * epi_words(NT),
                                                mw + r, mw + r + 16);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
  };
  if constexpr (EPI == EPI_GRAD) with_act(g.act, tiles);
  else tiles(std::integral_constant<int, ACT_SILU>{});
}

template <int KIND, int EPI, int W, int NB, int DT>
__global__ __launch_bounds__(256, W == 4 && NB == 2 ? 2 : 1) void large_kernel(TileArgs g, int n_tiles,
                                                                    int m_tiles, int per) {
  // one array for everything: with a second one in LDS the compiler waits for
  // all memory before LDS reads in the K loop
  __shared__ u32x4_t lds[LargeLds<KIND, EPI, W, NB>::WORDS16];
  large_body<KIND, EPI, W, NB, DT>(g, n_tiles, m_tiles, per, lds);
}

// ---------------------------------------------------------------- host side
// Tiles of a product with tiles of 32 W, in n (pairs of products: half as many
// columns) and m.
static int64_t tiles_of(int64_t m, int64_t n, bool pair, int w) {
  const int64_t rows = 32 * w, cols = pair ? 16 * w : 32 * w;
  return ((m + rows - 1) / rows) * ((n + cols - 1) / cols);
}

// Whether 256 x 256 tiles serve a product of codes better than 128 x 128 ones, by
// the time in us that its tiles take, st stages each: of the former a CU runs one, in
// rounds; of the latter two at once, or in the last round and where there are at
// most 256, one, with twice the stages in flight.  (us, 256 / 128: 4096 x 4096 x
// 11008 169 / 190, 1024 x 4096 x 11008 55 / 59; 2048 x 4096 x 8448 104 / 90, gated
// 4096 x 512 x 11008 141 / 110, 512 x 11008 x 4096 103 / 44.)
static bool large_tiles(int64_t m, int64_t n, bool pair, int64_t kb) {
  const int64_t t8 = tiles_of(m, n, pair, 8), t4 = tiles_of(m, n, pair, 4);
  const double st = (double)((kb + kStageBytes - 1) / kStageBytes);
  const double two = 2 * (0.43 * st + 3.6), one = 0.6 * st + 4;
  const int64_t last = t4 % 512;
  const double large = (double)((t8 + 255) / 256) * (1.17 * st + 17.7);
  const double small = 3 + (double)(t4 / 512) * two + (last == 0 ? 0 : last <= 256 ? one : two);
  return large <= small;
}

template <int KIND, int EPI, int W, int NB, int DT>
static hipError_t launch_w(const TileArgs& t, int64_t m, int64_t n, hipStream_t s) {
  constexpr int rows = 32 * W, cols = EPI == EPI_GATED || EPI == EPI_GRAD ? 16 * W : 32 * W;
  int64_t n_tiles = (n + cols - 1) / cols;
  const int64_t m_tiles = (m + rows - 1) / rows;
  int per = 0;
  if constexpr (EPI == EPI_PARTIAL) {
    per = (t.kb / kStageBytes + t.plan.splits - 1) / t.plan.splits;
    n_tiles *= t.plan.splits;
  }
  if (n_tiles * m_tiles > kMaxGroups) return hipErrorInvalidValue;
  return launch_kernel(large_kernel<KIND, EPI, W, NB, DT>, dim3((unsigned)(n_tiles * m_tiles)), dim3(256),
                       s, t, (int)n_tiles, (int)m_tiles, per);
}

template <int KIND, int EPI, int DT>
static hipError_t launch(const TileArgs& t, hipStream_t s) {
  // the gradient epilogue also writes the padding of its operands
  const int64_t n = EPI == EPI_GRAD ? t.Np : t.N;
  const int64_t m = EPI == EPI_GRAD && t.dt != nullptr ? t.Mp : t.M;
  constexpr bool pair = EPI == EPI_GATED || EPI == EPI_GRAD;
  if (large_tiles(m, n, pair, t.kb)) return launch_w<KIND, EPI, 8, 2, DT>(t, m, n, s);
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

// y = the sum of the partial products (fp16: times the row's factor), rounded once; 4
// columns per thread.
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
  for (int s = 0; s < t.plan.splits; ++s)
    v += *reinterpret_cast<const f32x4_t*>(t.part + s * (int64_t)t.M * ld + at);
  const float k = DT == XF16 ? t.sa[m] : 1.f;
  T* y = static_cast<T*>(second ? t.y2 : t.y) + (int64_t)mo * t.ldy + n;
  const float o[4] = {v[0] * k, v[1] * k, v[2] * k, v[3] * k};
  store4(y, o, min(4, t.N - n), vec4_ok(second ? t.y2 : t.y, t.ldy, 2));
}

// By the time in us that either way takes.  256 x 256 tiles, in rounds of 256, are the
// faster ones where many stages fill whole rounds (4096 x 4096 x 22016 contracted:
// 683 against 809 us, 8192 x 4096 x 11008 639 against 721); of 128 x 128 tiles two or
// more run on a CU, one's epilogue beside another's products, and the last of them
// are not waited for as long (22016 x 4096 x 512 131 against 178 us, 8192 x 8192 x
// 1024 145 against 167, 4096 x 11008 x 4096 331 against 342).  Where they leave CUs
// idle the contraction is split, at the price of writing and adding fp32 sums (128 x
// 4096 x 22016 254 -> 46 us with 16 shares, 2048 x 1024 x 14336 191 -> 92 with 4, 64
// x 2048 x 2048 33 -> 19 with 8; 2048 x 2048 x 300 not: 18 -> 32 with 2).
PlainPlan plain_plan(int64_t M, int64_t N, int64_t kb) {
  const int64_t all = kb / kStageBytes, t8 = tiles_of(M, N, false, 8), t4 = tiles_of(M, N, false, 4);
  const double large = (double)((t8 + 255) / 256) * (1.8 * (double)all + 9);
  PlainPlan p{8, 1};
  double best = large;
  for (int64_t s = 1; s <= 32 && (s == 1 || (t4 * s <= 512 && 3 * s <= all)); ++s) {
    // the same number of stages in all shares but the last, which is not empty
    const int64_t per = (all + s - 1) / s, shares = (all + per - 1) / per, wgs = t4 * shares;
    const double turns = wgs < 512 ? 2 : (double)wgs / 256;
    double us = wgs <= 256 ? 0.8 * (double)per + 2 : turns * (0.52 * (double)per + 1);
    if (shares > 1) us += 5 + (double)(shares * M * N) * 1e-6;
    if (us < best) best = us, p = PlainPlan{4, (int)shares};
  }
  return p;
}

template <int DT> static hipError_t tile_plain(const TileArgs& t, hipStream_t s) {
  if (t.plan.splits == 1)
    return t.plan.w == 8 ? launch_w<DT, EPI_PLAIN, 8, 2, DT>(t, t.M, t.N, s)
                         : launch_w<DT, EPI_PLAIN, 4, 2, DT>(t, t.M, t.N, s);
  TileArgs p = t;
  p.y = t.part;
  p.ldy = round_up(t.N, 4);
  p.y_dtype = YF32;
  const hipError_t e = launch_w<DT, EPI_PARTIAL, 4, 2, DT>(p, t.M, t.N, s);
  if (e != hipSuccess) return e;
  const int bpr = (t.N + 1023) / 1024;
  return launch_kernel(sum_partials_kernel<DT>, dim3((unsigned)((int64_t)t.M * bpr)), dim3(256), s, t, bpr);
}

hipError_t launch_tile_plain(const TileArgs& t, int dtype, hipStream_t s) {
  return dtype == XF16 ? tile_plain<XF16>(t, s) : tile_plain<XBF16>(t, s);
}

}  // namespace qmm
