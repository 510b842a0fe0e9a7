// mx4_large.hip -- products of microscaled 4-bit codes for more rows than a decode
// batch, on v_mfma_scale_f32_16x16x128_f8f6f4: the matrix cores take both operands' codes
// and scales as they are stored.
//
// Tiles of 256 x 256 (W = 8) or 128 x 128 (W = 4) by 4 waves as 2 x 2; a wave owns W x
// W tiles of 16 x 16, whose accumulators are pinned to the matrix-core (AGPR) registers.
//  * both operands are packed (chunks of 512 values of 16 rows).  A stage is half a chunk,
//    two MFMA k steps: 2 KiB of a strip as they lie in memory, by loads straight to LDS, read
//    from there as consecutive 256 bytes by 16 lanes.  NB stages are in flight;
//  * a lane's 4 scales of a chunk are one word of LDS, of which the instruction picks the
//    byte: one read for each operand and chunk;
//  * the operands of the next k step are read while the MFMAs of this one run.  When a
//    stage's second k step begins all of its operands are in registers, and one barrier
//    there does everything: the next stage has arrived, the one after next may go out;
//  * a workgroup stays for tile after tile: the last stages of one already load and read the
//    first of the next, and y leaves straight from the accumulators.
// Strips past M or N read zeros.
// 4096 x 4096 x 11008, bf16 y: 97 us, 3.8 PFLOP/s, at the power limit (78 with codes of 0, 4.7; the instruction alone from
// registers runs at 6.4 to 7.3 with random codes and 8.6 to 9.5 with zeros).
#include "mx4_device.h"
#include "w8a8_tile.h"

namespace qmm {

// s_waitcnt vmcnt(n) lgkmcnt(0)
static constexpr int wait_mem(int n) { return n > 63 ? wait_mem(63) : (n & 15) | ((n >> 4) << 14) | 0x0070; }

// Block J of a lane's 4: byte J of the scale words.
template <int J>
__device__ __forceinline__ void mfma_pinned_mx4(f32x4_t& c, const u32x4_t& a, const u32x4_t& b, uint32_t sa,
                                                uint32_t sb) {
#define QMM_MFMA(lo, hi)                                                                                     \
  asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[" #lo "," #lo ",0] op_sel_hi:[" #hi \
               "," #hi ",0] cbsz:4 blgp:4" : "+a"(c) : "v"(a), "v"(b), "v"(sa), "v"(sb))
  if constexpr (J == 0) QMM_MFMA(0, 0);
  else if constexpr (J == 1) QMM_MFMA(1, 0);
  else if constexpr (J == 2) QMM_MFMA(0, 1);
  else QMM_MFMA(1, 1);
#undef QMM_MFMA
}

// LDS of a workgroup in 16-byte words: NB stages of both operands' codes, and the scales of
// their NB / 2 chunks.
template <int W, int NB> struct Mx4LargeLds {
  static constexpr int CODES = 32 * W * 8;  // of one operand and stage
  static constexpr int STAGE = 2 * CODES;
  static constexpr int SCALES = 32 * W;     // of one operand and chunk: a word of 4 for each of 64 lanes of a strip
  static constexpr int WORDS16 = NB * STAGE + NB * SCALES;
};

// Exchanges the odd rows of 16 lanes of a with the even rows of b: a is then its own row 0,
// b's row 0, its own row 2, b's row 2, and b is a's row 1, its own 1, a's 3, its own 3.
__device__ __forceinline__ void rows_swap(uint32_t (&a)[2], uint32_t (&b)[2]) {
  asm volatile("s_nop 1\n\tv_permlane16_swap_b32 %0, %2\n\tv_permlane16_swap_b32 %1, %3"
               : "+v"(a[0]), "+v"(a[1]), "+v"(b[0]), "+v"(b[1]));
}

// (a device function beside its kernel: the host pass drops a kernel whose own
// body has matrix-core registers in inline asm)
template <int W, int NB, class Y>
__device__ __forceinline__ void mx4_large_body(const Mx4Args& g, int n_tiles, int m_tiles, int groups, u32x4_t* lds) {
  typedef Mx4LargeLds<W, NB> L;
  constexpr int TILE = 32 * W, PIECES = W / 2, NC = NB / 2;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, quad = lane >> 4;
  const int wm = wave >> 1, wn = wave & 1;
  const int chunks = mx4_chunks(g.K);
  const int strip_bytes = (int)mx4_strip_bytes(g.K);
  const int total = n_tiles * m_tiles;

  // What is loaded next: chunk q of tile `item`, by buffers of this wave's W / 2 strips of either
  // operand from that chunk on (of a tile that does not exist: empty ones).
  int item = (int)blockIdx.x, q = 0;
  const uint8_t *pa, *pb;
  uint32_t na, nb;
  auto strips_of = [&](const uint8_t* w, int first, int limit, const uint8_t*& p, uint32_t& bytes) {
    const int n = min(PIECES, limit - first);
    p = w + (int64_t)(n > 0 ? first : 0) * strip_bytes;
    bytes = n > 0 ? (uint32_t)(n * strip_bytes) : 0u;
  };
  auto open_item = [&]() {
    int mt = 0, nt = 0;
    const bool ok = item < total;
    if (ok) tile_of(item, n_tiles, m_tiles, &mt, &nt);
    strips_of(g.a, (mt * TILE) / 16 + PIECES * wave, ok ? (g.M + 15) / 16 : 0, pa, na);
    strips_of(g.w, (nt * TILE) / 16 + PIECES * wave, ok ? (g.N + 15) / 16 : 0, pb, nb);
  };
  auto next_chunk = [&]() {
    if (++q < chunks) {
      // (a strip's chunk lies within what its buffer holds from the strip on: only whole strips can be missing)
      pa += kChunkBytes;
      pb += kChunkBytes;
      return;
    }
    q = 0;
    item += groups;
    open_item();
  };
  // (the lane's offset says whether its strip exists; what is added to it stays within the strip)
  int off[PIECES];
#pragma unroll
  for (int i = 0; i < PIECES; ++i) off[i] = i * strip_bytes + 16 * lane;
  const int soff = (lane >> 4) * strip_bytes + 4096 + 16 * l16;  // 16 lanes on a strip's scales
  auto lds_at = [&](int word) { return (__attribute__((address_space(3))) void*)(lds + word); };
  // load j of this wave's share of that chunk's stage h, to chunk buffer `cb`: 2 KiB of each strip, and with
  // the first stage the scales
  constexpr int LOADS[2] = {2 * W + 2, 2 * W};
  auto load = [&](int j, int h, int cb) {
    const int base = (2 * cb + h) * L::STAGE;
    if (j < 2 * W) {
      const int o = j / W, i = j % W;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(make_buf(o == 0 ? pa : pb, o == 0 ? na : nb),
                                               lds_at(base + o * L::CODES + (W * wave + i) * 64), 16, off[i / 2],
                                               1024 * (2 * h + i % 2), 0, 0);
    } else {
      const int o = j - 2 * W;
      if (W == 8 || lane < 32)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(make_buf(o == 0 ? pa : pb, o == 0 ? na : nb),
                                                 lds_at(NB * L::STAGE + (2 * cb + o) * L::SCALES + 16 * PIECES * wave), 16,
                                                 soff, 0, 0, 0);
    }
  };
  // operand i (W of A, then W of B) of k step k of stage h of chunk buffer cb
  const int oa = 128 * W * wm + lane, ob = L::CODES + 128 * W * wn + lane;
  auto frag = [&](int i, int k, int h, int cb) {
    return lds[(2 * cb + h) * L::STAGE + (i < W ? oa + 128 * i : ob + 128 * (i - W)) + 64 * k];
  };
  // its 4 scales
  auto scale = [&](int i, int cb) {
    const uint32_t* s = reinterpret_cast<const uint32_t*>(lds + NB * L::STAGE + (2 * cb + (i < W ? 0 : 1)) * L::SCALES);
    return s[64 * (i < W ? W * wm + i : W * wn + i - W) + lane];
  };

  u32x4_t f[2][2 * W];  // operands of the two k steps
  uint32_t sc[2 * W], sn[2 * W];
  open_item();
#pragma unroll
  for (int c = 0; c < NC; ++c) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < LOADS[h]; ++j) load(j, h, c);
    next_chunk();
  }
  __builtin_amdgcn_s_waitcnt(wait_mem(NC == 1 ? LOADS[1] : LOADS[1] + LOADS[0] + LOADS[1]));
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2 * W; ++i) f[0][i] = frag(i, 0, 0, 0), sc[i] = scale(i, 0);
  int cb = 0;
  bool stored = false;  // the tile before left in STORES stores a wave
  constexpr int STORES = sizeof(Y) == 4 ? W * W : W * W / 2;

#pragma unroll 1
  for (int b = (int)blockIdx.x; b < total; b += groups) {
    f32x4_t acc[W][W];
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
      for (int s = 0; s < W; ++s) acc[i][s] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    __builtin_amdgcn_sched_barrier(0);

#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
      const int cn = NC == 1 ? 0 : cb ^ 1;  // the next chunk's buffer
      // k step 2 h + k = j: groups of 4 MFMAs, between them the reads of the next step's operands (in the order
      // of their first use; with the last step the next chunk's scales) and, in a stage's second step, the loads
      // that follow it into its buffer.  Past a tile's last chunk all go on with the next tile's first.
      auto step = [&](auto jc) {
        constexpr int j = decltype(jc)::value, h = j / 2, k = j % 2;
        constexpr int GROUPS = W * W / 4, READS = 2 * W;
        // reads: in a first step all are back before the barrier
        constexpr int READ_GROUPS = k == 0 ? GROUPS - GROUPS / 8 : GROUPS;
        constexpr int LOAD_GROUPS = GROUPS;
#pragma unroll
        for (int t = 0; t < GROUPS; ++t) {
#pragma unroll
          for (int o = min(READS, t * READS / READ_GROUPS); o < min(READS, (t + 1) * READS / READ_GROUPS); ++o) {
            const int i = o == 0 ? 0 : (o <= W ? W + o - 1 : o - W);
            if constexpr (k == 0) f[1][i] = frag(i, 1, h, cb);
            else f[0][i] = h == 0 ? frag(i, 0, 1, cb) : frag(i, 0, 0, cn);
            if (j == 3) sn[i] = scale(i, cn);
          }
          if (k == 1) {
#pragma unroll
            for (int l = min(LOADS[h], t * LOADS[h] / LOAD_GROUPS); l < min(LOADS[h], (t + 1) * LOADS[h] / LOAD_GROUPS); ++l)
              load(l, h, cb);
          }
          // (two wait states between a vector instruction's result, such as a copied scale or a
          // cleared accumulator, and the matrix instruction that reads it: the compiler sees none here)
          if (t == 0) asm volatile("s_nop 1" ::: "memory");
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const int i = (4 * t + s) / W, n = (4 * t + s) % W;
            // B's columns are the rows of the product: a lane then holds 4 consecutive columns of one row of y
            mfma_pinned_mx4<j>(acc[i][n], f[k][W + n], f[k][i], sc[W + n], sc[i]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (k == 0) {
          // the next stage has arrived: loads return in order, and so do the stores that the last tile
          // left after this stage's loads
          constexpr int later = NC == 1 ? 0 : LOADS[0] + LOADS[1];
          if (h == 0 && stored) __builtin_amdgcn_s_waitcnt(wait_mem(later + STORES));
          else __builtin_amdgcn_s_waitcnt(wait_mem(later));
          __syncthreads();
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      step(std::integral_constant<int, 0>{});
      step(std::integral_constant<int, 1>{});
      step(std::integral_constant<int, 2>{});
      step(std::integral_constant<int, 3>{});
      stored = false;
      next_chunk();
#pragma unroll
      for (int i = 0; i < 2 * W; ++i) sc[i] = sn[i];
      cb = cn;
    }
    // the accumulators were last written by MFMAs that the compiler does not see
    // as such: give them their latency, then pass each through an empty asm
    // ordered after that, so that no read of one moves above it
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
      for (int s = 0; s < W; ++s) asm volatile("" : "+a"(acc[i][s]));
    __builtin_amdgcn_sched_barrier(0);

    // Straight from the registers: a lane holds columns 16 c + 4 quad .. + 3 of row l16 of each tile.
    int mt, nt;
    tile_of(b, n_tiles, m_tiles, &mt, &nt);
    const int m = mt * TILE + 16 * W * wm + l16, n0 = nt * TILE + 16 * W * wn;
    Y* y = static_cast<Y*>(g.y) + (int64_t)m * g.ldy + n0;
    const int64_t down = 16 * g.ldy;
    const bool whole = (mt + 1) * (int64_t)TILE <= g.M && (nt + 1) * (int64_t)TILE <= g.N;
    // f(first column, values) for what a lane stores of row tile i: 16 bytes, of which 4 lanes make 64
    // consecutive ones
    constexpr int PER = 16 / (int)sizeof(Y);
    auto pieces = [&](int i, auto&& put) {
      if constexpr (sizeof(Y) == 4) {
#pragma unroll
        for (int c = 0; c < W; ++c) put(16 * c + 4 * quad, __builtin_bit_cast(u32x4_t, acc[i][c]));
      } else {
        // two neighbouring strips exchange rows of lanes, so that a lane has 8 columns of one
#pragma unroll
        for (int c = 0; c < W; c += 2) {
          typedef Y Y2 __attribute__((ext_vector_type(2)));
          uint32_t v[2][2];
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const Y2 p = {(Y)acc[i][c + s][2 * j], (Y)acc[i][c + s][2 * j + 1]};
              v[s][j] = __builtin_bit_cast(uint32_t, p);
            }
          rows_swap(v[0], v[1]);
          put(16 * (c + (quad & 1)) + 8 * (quad >> 1), u32x4_t{v[0][0], v[0][1], v[1][0], v[1][1]});
        }
      }
    };
    typedef u32x4_t __attribute__((aligned(2))) out_t;  // rows start anywhere
    // (the two branches read the accumulators behind different asm: read before the branch, all of them at
    // once, they would not fit the vector registers)
    if (whole) {
#pragma unroll
      for (int i = 0; i < W; ++i) {
#pragma unroll
        for (int c = 0; c < W; ++c) asm volatile("; whole" : "+a"(acc[i][c]));
        pieces(i, [&](int n, u32x4_t v) { *reinterpret_cast<out_t*>(y + n) = v; });
        y += down;
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
#pragma unroll
        for (int c = 0; c < W; ++c) asm volatile("; edge" : "+a"(acc[i][c]));
        pieces(i, [&](int n, u32x4_t v) {
          const int left = m + 16 * i < g.M ? g.N - (n0 + n) : 0;  // columns of this row that exist
          if (left >= PER) {
            *reinterpret_cast<out_t*>(y + n) = v;
          } else if (left > 0) {
#pragma unroll 1
            for (int j = 0; j < left; ++j) {
              if constexpr (sizeof(Y) == 4) {
                const uint32_t e = v[0];
                y[n + j] = __builtin_bit_cast(float, e);
                v = u32x4_t{v[1], v[2], v[3], 0u};
              } else {
                y[n + j] = __builtin_bit_cast(Y, (uint16_t)v[0]);
                v = u32x4_t{(v[0] >> 16) | (v[1] << 16), (v[1] >> 16) | (v[2] << 16), (v[2] >> 16) | (v[3] << 16), v[3] >> 16};
              }
            }
          }
        });
        y += down;
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    stored = whole;
  }
}

template <int W, int NB, class Y>
__global__ __launch_bounds__(256, W == 4 && NB == 2 ? 2 : 1) void mx4_large_kernel(Mx4Args g, int n_tiles, int m_tiles,
                                                                                   int groups) {
  // one array for everything: with a second one in LDS the compiler waits for
  // all memory before LDS reads in the K loop
  __shared__ u32x4_t lds[Mx4LargeLds<W, NB>::WORDS16];
  mx4_large_body<W, NB, Y>(g, n_tiles, m_tiles, groups, lds);
}

// ---------------------------------------------------------------- host side
static int64_t tiles(int64_t m, int64_t n, int w) {
  return ((m + 32 * w - 1) / (32 * w)) * ((n + 32 * w - 1) / (32 * w));
}

template <int W, int NB, class Y> static hipError_t launch_y(const Mx4Args& a, hipStream_t s) {
  const int n_tiles = (int)(((int64_t)a.N + 32 * W - 1) / (32 * W)), m_tiles = (int)(((int64_t)a.M + 32 * W - 1) / (32 * W));
  const int64_t total = (int64_t)n_tiles * m_tiles;
  if (total > INT32_MAX / 2) return hipErrorInvalidValue;
  const int most = W == 4 && NB == 2 ? 512 : 256;  // workgroups at once
  const int groups = total < most ? (int)total : most;
  return launch_kernel(mx4_large_kernel<W, NB, Y>, dim3((unsigned)groups), dim3(256), s, a, n_tiles, m_tiles, groups);
}
template <int W, int NB> static hipError_t launch_w(const Mx4Args& a, hipStream_t s) {
  switch (a.y_dtype) {
    case XF16: return launch_y<W, NB, _Float16>(a, s);
    case XBF16: return launch_y<W, NB, __bf16>(a, s);
  }
  return launch_y<W, NB, float>(a, s);
}

// 256 x 256 from three quarters of a round of them on, else 128 x 128, of which one a CU keeps 4 stages in flight and two a CU 2
// (K = 4096, us from codes, 256, 128 with 4 stages and with 2: 512 x 11008, 86 tiles of 256, 33.7, 29.2, 24.3; 1024 x 11008, 172,
// 35.4, 41.1, 36.8; 1536 x 8192, 192, 37.1, 42.5, 38.7; 2048 x 8192, 256, 41.9, 53.3, 45.7; 256 x 4096, 64 of 128, 34.4, 20.3, 21.1).
hipError_t launch_mx4_large(const Mx4Args& a, hipStream_t s) {
  if (tiles(a.M, a.N, 8) >= 192) return launch_w<8, 2>(a, s);
  return tiles(a.M, a.N, 4) <= 256 ? launch_w<4, 4>(a, s) : launch_w<4, 2>(a, s);
}

}  // namespace qmm
