// mx4_large.hip -- products of microscaled 4-bit codes for more rows than a decode
// batch, on v_mfma_scale_f32_16x16x128_f8f6f4: the matrix cores take both operands' codes
// and scales as they are stored.
//
// Tiles of 256 x 256 (W = 8) or 128 x 128 (W = 4) by 4 waves as 2 x 2; a wave owns W x
// W tiles of 16 x 16, whose accumulators are pinned to the matrix-core (AGPR) registers.
//  * a stage is 256 values of K, two MFMA k steps: 2 KiB of a strip's codes and 128 bytes of
//    scales.  Both operands' codes and scales go to LDS by loads straight to it, NB
//    stages in flight;
//  * both operands are packed: 1 KiB of a strip as it lies in memory, read from LDS as
//    consecutive 256 bytes by 16 lanes;
//  * a lane's block in k step k is 2 (lane / 16) + k of the stage's 8: the scales of both k
//    steps are then neighbouring bytes, one 2-byte read for each operand and stage, of
//    which the instruction picks the byte;
//  * the operands of the next k step are read while the MFMAs of this one run.  When a
//    stage's second k step begins all of its operands are in registers, and one barrier
//    there does everything: the next stage has arrived, the one after may go out.
// Strips past M or N and steps past K read zeros.
#include "mx4_device.h"
#include <stdlib.h>
#include "w8a8_tile.h"

namespace qmm {

static constexpr int wait_mem(int n) { return (n & 15) | ((n >> 4) << 14) | 0x0070; }

// k step K of a stage: byte K of the scale words.
template <int K>
__device__ __forceinline__ void mfma_pinned_mx4(f32x4_t& c, const u32x4_t& a, const u32x4_t& b, uint32_t sa,
                                                uint32_t sb) {
  if constexpr (K == 0)
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[0,0,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                 : "+a"(c) : "v"(a), "v"(b), "v"(sa), "v"(sb));
  else
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                 : "+a"(c) : "v"(a), "v"(b), "v"(sa), "v"(sb));
}

// LDS of a workgroup in 16-byte words: NB stages of both operands' codes and scales, and in
// their place later the epilogue's tiles.
template <int W, int NB> struct Mx4LargeLds {
  static constexpr int CODES = 32 * W * 8;                 // of one operand and stage
  static constexpr int SCALES = 32 * W / 2;                // 8 bytes a row
  static constexpr int STAGE = 2 * (CODES + SCALES);
  static constexpr int G = 4;                              // row tiles of a wave in LDS at once
  static constexpr int EPI = G * epi_words(W);             // words of a wave
  static constexpr int WORDS16 = NB * STAGE > EPI ? NB * STAGE : EPI;
};

// (a device function beside its kernel: the host pass drops a kernel whose own
// body has matrix-core registers in inline asm)
template <int W, int NB>
__device__ __forceinline__ void mx4_large_body(const Mx4Args& g, int n_tiles, int m_tiles, u32x4_t* lds) {
  typedef Mx4LargeLds<W, NB> L;
  constexpr int TILE = 32 * W, STAGE = L::STAGE, PIECES = W / 2;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, quad = lane >> 4;
  int mt, nt;
  tile_of((int)blockIdx.x, n_tiles, m_tiles, &mt, &nt);
  const int m0 = mt * TILE, n0 = nt * TILE;
  const int wm = wave >> 1, wn = wave & 1;
  const int steps = mx4_steps(g.K), nst = (steps + 1) / 2;
  const int strip_bytes = (int)mx4_strip_bytes(g.K);

  // This wave's W / 2 strips of either operand, each a buffer that ends with the last.
  auto strips_of = [&](const uint8_t* p, int first, int limit) {
    const int n = min(PIECES, limit - first);
    return make_buf(p + (int64_t)(n > 0 ? first : 0) * strip_bytes, n > 0 ? (uint32_t)(n * strip_bytes) : 0u);
  };
  const buf_t ra = strips_of(g.a, m0 / 16 + PIECES * wave, (g.M + 15) / 16);
  const buf_t rb = strips_of(g.w, n0 / 16 + PIECES * wave, (g.N + 15) / 16);

  // Lanes' offsets: 16 bytes of codes; scales 4 bytes a lane, dword d of the wave's, row d / 2
  constexpr int SL = W / 4;  // loads of one operand's scales (128 W / 4 bytes a wave)
  int so[SL];
#pragma unroll
  for (int i = 0; i < SL; ++i) {
    const int d = 64 * i + lane, r = d >> 1;
    so[i] = (r >> 4) * strip_bytes + 1024 * steps + 16 * (r & 15) + 4 * (d & 1);
  }
  constexpr int LOADS = 2 * W + 2 * SL;
  auto lds_at = [&](int word) { return (__attribute__((address_space(3))) void*)(lds + word); };
  // load j of this wave's share of stage st (past the last stage: the last again, unused)
  auto load = [&](int j, int st) {
    const int base = st % NB * STAGE;
    const int q = min(st, nst - 1);
    if (j < 2 * W) {
      // strip i's step 2 q + h; past K nothing
      const int o = j / W, i = j % W / 2, h = j % 2, step = 2 * q + h;
      const int at = step < steps ? i * strip_bytes + 1024 * step : 0x7FFF0000;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(o == 0 ? ra : rb, lds_at(base + o * L::CODES + (W * wave + j % W) * 64), 16,
                                               16 * lane + at, 0, 0, 0);
    } else {
      const int o = (j - 2 * W) / SL, i = (j - 2 * W) % SL;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(o == 0 ? ra : rb, lds_at(base + 2 * L::CODES + o * L::SCALES + (SL * wave + i) * 16),
                                               4, so[i] + 256 * (q >> 1) + 8 * (q & 1), 0, 0, 0);
    }
  };
  // operand i (W of A, then W of B) of k step k of stage st
  const int oa = 128 * W * wm + l16, ob = L::CODES + 128 * W * wn + l16;
  auto frag = [&](int i, int k, int st) {
    return lds[st % NB * STAGE + (i < W ? oa + 128 * i : ob + 128 * (i - W)) + 16 * (2 * quad + k)];
  };
  // both k steps' scales of operand i
  const int os = 16 * W * wm + l16, ot = 16 * W * wn + l16;
  auto scale = [&](int i, int st) {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(lds + st % NB * STAGE + 2 * L::CODES + (i < W ? 0 : L::SCALES));
    return (uint32_t)p[4 * (i < W ? os + 16 * i : ot + 16 * (i - W)) + quad];
  };

  f32x4_t acc[W][W];
#pragma unroll
  for (int i = 0; i < W; ++i)
#pragma unroll
    for (int s = 0; s < W; ++s) acc[i][s] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  u32x4_t f[2][2 * W];  // operands of the two k steps
  uint32_t sc[2 * W], sn[2 * W];
#pragma unroll
  for (int q = 0; q < NB; ++q)
#pragma unroll
    for (int j = 0; j < LOADS; ++j) load(j, q);
  __builtin_amdgcn_s_waitcnt(wait_mem((NB - 1) * LOADS));
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2 * W; ++i) f[0][i] = frag(i, 0, 0), sc[i] = scale(i, 0);

#pragma unroll 1
  for (int st = 0; st < nst; ++st) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      // groups of 4 MFMAs; the next k step's operands (and scales) are read in the first half
      // of them, in the order of their first use; in the second k step the loads go out
      constexpr int GROUPS = W * W / 4, PER = 4 * W / GROUPS;
#pragma unroll
      for (int t = 0; t < GROUPS; ++t) {
        if (t < GROUPS / 2) {
#pragma unroll
          for (int h = 0; h < PER; ++h) {
            const int q = PER * t + h, i = q == 0 ? 0 : (q <= W ? W + q - 1 : q - W);
            f[k ^ 1][i] = frag(i, k ^ 1, st + k);
            if (k == 1) sn[i] = scale(i, st + 1);
          }
        }
        if (k == 1) {
#pragma unroll
          for (int j = t * LOADS / GROUPS; j < (t + 1) * LOADS / GROUPS; ++j) load(j, st + NB);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int i = (4 * t + s) / W, c = (4 * t + s) % W;
          if (k == 0) mfma_pinned_mx4<0>(acc[i][c], f[k][i], f[k][W + c], sc[i], sc[W + c]);
          else mfma_pinned_mx4<1>(acc[i][c], f[k][i], f[k][W + c], sc[i], sc[W + c]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (k == 0) {
        __builtin_amdgcn_s_waitcnt(wait_mem((NB - 2) * LOADS));
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int i = 0; i < 2 * W; ++i) sc[i] = sn[i];
  }
  __builtin_amdgcn_s_waitcnt(wait_mem(0));
  __syncthreads();  // every wave has left the stages: their LDS becomes the epilogue's
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

  uint32_t* t0 = reinterpret_cast<uint32_t*>(lds) + wave * L::EPI;
  TileArgs ge{};
  ge.y = g.y, ge.y2 = nullptr, ge.y_dtype = g.y_dtype, ge.ldy = g.ldy;
  ge.M = g.M, ge.N = g.N, ge.M2 = g.M, ge.Mv = g.M;
  Epilogue<XBF16, EPI_PLAIN, W, XBF16> epi;
  epi.init(ge, n0 + 16 * W * wn, lane);
#pragma unroll
  for (int h = 0; h < W / L::G; ++h) {
#pragma unroll
    for (int i = 0; i < L::G; ++i) put_tile<XBF16, W>(acc[h * L::G + i], t0 + i * epi_words(W), lane);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll 1
    for (int i = 0; i < L::G; ++i) {
      const int m = m0 + 16 * W * wm + 16 * (h * L::G + i);
      epi.template tile<ACT_SILU>(ge, t0 + i * epi_words(W), nullptr, nullptr, m, m + 16);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

template <int W, int NB>
__global__ __launch_bounds__(256, W == 4 && NB == 2 ? 2 : 1) void mx4_large_kernel(Mx4Args g, int n_tiles, int m_tiles) {
  // one array for everything: with a second one in LDS the compiler waits for
  // all memory before LDS reads in the K loop
  __shared__ u32x4_t lds[Mx4LargeLds<W, NB>::WORDS16];
  mx4_large_body<W, NB>(g, n_tiles, m_tiles, lds);
}

// ---------------------------------------------------------------- host side
static int64_t tiles(int64_t m, int64_t n, int w) {
  return ((m + 32 * w - 1) / (32 * w)) * ((n + 32 * w - 1) / (32 * w));
}

template <int W, int NB> static hipError_t launch_w(const Mx4Args& a, hipStream_t s) {
  const int n_tiles = (int)(((int64_t)a.N + 32 * W - 1) / (32 * W)), m_tiles = (a.M + 32 * W - 1) / (32 * W);
  if ((int64_t)n_tiles * m_tiles > kMaxGroups) return hipErrorInvalidValue;
  return launch_kernel(mx4_large_kernel<W, NB>, dim3((unsigned)(n_tiles * m_tiles)), dim3(256), s, a, n_tiles, m_tiles);
}

hipError_t launch_mx4_large(const Mx4Args& a, hipStream_t s) {
  const char* e = getenv("MX4_W");
  const int force = e ? atoi(e) : 0;
  if (force == 8 || (force == 0 && tiles(a.M, a.N, 8) >= 192)) return launch_w<8, 2>(a, s);
  return (force == 44 || (force == 0 && tiles(a.M, a.N, 4) <= 256)) ? launch_w<4, 4>(a, s) : launch_w<4, 2>(a, s);
}

}  // namespace qmm
