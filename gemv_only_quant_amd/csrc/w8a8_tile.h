// w8a8_tile.h -- what the matrix-core kernels of the int8 x int8 operators
// share: accumulators, the order of tiles, and the epilogues.
#pragma once
#include <type_traits>

#include "w8a8_device.h"

namespace qmm {

enum { EPI_SCALE = 0, EPI_GATED = 1, EPI_GRAD = 2, EPI_PLAIN = 3, EPI_PARTIAL = 4 };

// KIND: kTypeI8, XF16 or XBF16
template <int KIND> struct Acc { typedef f32x4_t type; };
template <> struct Acc<kTypeI8> { typedef i32x4_t type; };

// LDS of the epilogue: a 16-row tile of a wave is 16 rows of 16 NT words,
// column c of row r at word c ^ 16 (r / 4 % (NT % 4 ? 2 : 4)): the four row
// quads that the accumulators hold at once then lie in different banks, and 4
// consecutive columns stay together.
template <int NT> __device__ __forceinline__ constexpr int epi_word(int row, int col) {
  return row * 16 * NT + (col ^ (16 * ((row >> 2) & (NT % 4 ? 1 : 3))));
}
constexpr int epi_words(int nt) { return 256 * nt; }
// ... and after the tiles, for the gradient epilogue, 64 rows transposed, of
// 16-bit values: a column's 64 rows are 128 bytes, 8 chunks, chunk c of column n
// at c ^ (n / 4 % 8), so that a wave's stores of one row pair meet two to a bank.
constexpr int epi_t_words(int nt) { return 16 * nt * 32; }

// Accumulators of a 16-row tile to its LDS.
template <int KIND, int NT>
__device__ __forceinline__ void put_tile(const typename Acc<KIND>::type (&acc)[NT], uint32_t* t0,
                                         int lane) {
  const int l16 = lane & 15, quad = lane >> 4;
#pragma unroll
  for (int s = 0; s < NT; ++s)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      // through a value: a bit cast of the vector's element itself takes
      // element 0 whatever r is, with this compiler
      const auto e = acc[s][r];
      t0[epi_word<NT>(4 * quad + r, 16 * s + l16)] = __builtin_bit_cast(uint32_t, e);
    }
}

// The epilogues, for a lane's 4 consecutive columns of the wave's output in
// rows that lie 64 / (columns / 4) apart.  What does not change from tile to
// tile (column scales, alignment) is read once, in init; the rows' scales are
// taken from LDS (`sa`, the workgroup's rows) and the gradient's incoming
// values one tile ahead: nothing in the loop over tiles waits for memory.
template <int KIND, int EPI, int NT, int DT> struct Epilogue {
  static constexpr bool PAIR = EPI == EPI_GATED || EPI == EPI_GRAD;
  static constexpr int COLS = PAIR ? 8 * NT : 16 * NT;  // output columns of the wave
  static constexpr int LPR = COLS / 4;                  // lanes per row
  static constexpr int RPP = 64 / LPR;                  // rows per pass
  static constexpr int PASSES = 16 / RPP;
  typedef typename Acc<KIND>::type acc_t;
  typedef typename Half16<DT>::type T;
  typedef T T4 __attribute__((ext_vector_type(4)));

  // row of this lane in pass p: in the gradient epilogue two passes take
  // neighbouring rows
  __device__ __forceinline__ int row_of(int p) const {
    return EPI == EPI_GRAD ? 2 * RPP * (p / 2) + 2 * (lane / LPR) + p % 2 : RPP * p + lane / LPR;
  }

  int lane, col, n0, n, nn;  // nn: columns of this lane that exist (may be <= 0)
  float s0[4], s1[4];        // column scales; of the up projection
  bool vec;
  uint16_t dh[EPI == EPI_GRAD ? PASSES : 1][4];  // the next tile's incoming gradient
  uint32_t levels[2][4];     // GRAD, fp16: of dg's and du's columns, a byte for each of 4 tiles

  __device__ __forceinline__ void init(const TileArgs& g, int n0_, int lane_) {
    lane = lane_, n0 = n0_;
    col = 4 * (lane % LPR), n = n0 + col, nn = min(4, g.N - n);
    if constexpr (EPI != EPI_PLAIN && EPI != EPI_PARTIAL) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s0[j] = j < nn ? g.sb[0][n + j] : 0.f;
        s1[j] = PAIR && j < nn ? g.sb[1][n + j] : 0.f;
      }
    }
    if constexpr (EPI == EPI_GRAD) {
      vec = vec4_ok(g.dh, g.lddh, 2);
    } else {
      vec = vec4_ok(g.y, g.ldy, g.y_dtype == YF32 ? 4 : 2) && (EPI != EPI_PLAIN || vec4_ok(g.y2, 0, 2));
    }
  }

  // The power of two of column j's 16 rows in this tile, whose level joins the others'
  // (fp16; else 1).
  __device__ __forceinline__ float block_power(const float (&v)[PASSES][4], int j, uint32_t& l, int part) {
    if constexpr (DT != XF16) return 1.f;
    float top = 0.f;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) top = fmaxf(top, fabsf(v[p][j]));
    if (LPR == 8) top = dpp_max<0x128>(top);  // row_ror:8
    const uint32_t level = level_of(rows4_max(top));
    l = part == 0 ? level : l | (level << (8 * part));
    return level_power(level);
  }

  // Requests what the tile at row m0 will need from memory.
  __device__ __forceinline__ void fetch(const TileArgs& g, int m0) {
    if constexpr (EPI == EPI_GRAD) {
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int m = m0 + row_of(p);
        const uint16_t* src = static_cast<const uint16_t*>(g.dh) + (int64_t)m * g.lddh + n;
        const bool row = m < g.M;
        if (vec && row && nn >= 4) {
          const u32x2_t q = *reinterpret_cast<const u32x2_t*>(src);
#pragma unroll
          for (int j = 0; j < 4; ++j) dh[p][j] = (uint16_t)(q[j / 2] >> (16 * (j % 2)));
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) dh[p][j] = row && j < nn ? src[j] : (uint16_t)0;
        }
      }
    }
  }

  // The tile that put_tile wrote to t0, whose first row is m0; sa: its rows'
  // scales; tt: the wave's transposed rows (GRAD), which leave with every fourth
  // tile (m0 from a multiple of 64 on); m1: the next tile's first row; ACT: the
  // activation (GRAD).
  template <int ACT>
  __device__ __forceinline__ void tile(const TileArgs& g, const uint32_t* t0, const float* sa,
                                       uint32_t* ttw, int m0, int m1) {
    if constexpr (EPI == EPI_PARTIAL) {
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int row = RPP * p + lane / LPR, m = m0 + row;
        const acc_t c = *reinterpret_cast<const acc_t*>(t0 + epi_word<NT>(row, col));
        // rows of whole 4 columns: ldy is a multiple of 4 and reaches past N
        if (m < g.M && nn > 0) *reinterpret_cast<acc_t*>(static_cast<float*>(g.y) + (int64_t)m * g.ldy + n) = c;
      }
    } else if constexpr (EPI == EPI_SCALE || EPI == EPI_PLAIN || EPI == EPI_GATED) {
      float v[PASSES][4];
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int row = RPP * p + lane / LPR;
        const acc_t c = *reinterpret_cast<const acc_t*>(t0 + epi_word<NT>(row, col));
        if constexpr (EPI == EPI_PLAIN) {
          const float k = DT == XF16 ? sa[row] : 1.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) v[p][j] = c[j] * k;
        } else if constexpr (EPI == EPI_SCALE) {
          const float a = sa[row];
#pragma unroll
          for (int j = 0; j < 4; ++j) v[p][j] = (float)c[j] * (a * s0[j]);
        } else {
          const acc_t u = *reinterpret_cast<const acc_t*>(t0 + epi_word<NT>(row, COLS + col));
          const float a = sa[row];
          with_act(g.act, [&](auto act) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float d;
              v[p][j] = act_parts<decltype(act)::value>((float)c[j] * (a * s0[j]), &d) *
                        ((float)u[j] * (a * s1[j]));
            }
          });
        }
      }
      with_y(g.y, g.y_dtype, [&](auto* yt) {
        typedef typename std::remove_pointer<decltype(yt)>::type Y;
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
          const int m = m0 + RPP * p + lane / LPR;
          if (m >= g.M || nn <= 0) continue;
          if constexpr (EPI == EPI_PLAIN) {
            const bool second = m >= g.M2;
            const int mo = second ? m - g.M2 : m;
            Y* yo = second ? static_cast<Y*>(g.y2) : yt;
            if (mo < g.Mv) store4(yo + (int64_t)mo * g.ldy + n, v[p], nn, vec);
          } else {
            store4(yt + (int64_t)m * g.ldy + n, v[p], nn, vec);
          }
        }
      });
    } else {
      // dg and du in fp32, then d = (dg sg | du su) row-major and dt = (dg sx | du sx)
      // transposed through LDS, zeros where a row or column only pads; in fp16 each
      // block of both times its power of two
      T* dd = static_cast<T*>(g.d);
      float dg[PASSES][4], du[PASSES][4];
#pragma unroll
      for (int p = 0; p < PASSES; ++p)
#pragma unroll
        for (int j = 0; j < 4; ++j) dg[p][j] = (float)__builtin_bit_cast(T, (uint16_t)dh[p][j]);
      fetch(g, m1);
      const int part = (m0 / 16) % 4;  // of the 64 transposed rows
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int row = row_of(p), m = m0 + row;
        const acc_t cg = *reinterpret_cast<const acc_t*>(t0 + epi_word<NT>(row, col));
        const acc_t cu = *reinterpret_cast<const acc_t*>(t0 + epi_word<NT>(row, COLS + col));
        const float a = sa[row];  // 0 for rows past M
        float vg[4], vu[4], top = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float gv = (float)cg[j] * (a * s0[j]), uv = (float)cu[j] * (a * s1[j]);
          float da;
          const float r = act_parts<ACT>(gv, &da);
          // rows past M and columns past N only pad: zeros, whatever the
          // scales are
          const bool ok = j < nn && m < g.M;
          const float e = dg[p][j];
          dg[p][j] = ok ? e * uv * da : 0.f;
          du[p][j] = ok ? e * r : 0.f;
          vg[j] = ok ? dg[p][j] * s0[j] : 0.f;
          vu[j] = ok ? du[p][j] * s1[j] : 0.f;
          if constexpr (DT == XF16) top = fmaxf(fmaxf(top, fabsf(vg[j])), fabsf(vu[j]));
        }
        const bool own = m < g.M && n < g.Np;  // n is a multiple of 4 and Np of 64
        float k = 1.f;
        if constexpr (DT == XF16) {
          const uint32_t level = level_of(lanes_max<kLevelD / 4>(top));
          k = level_power(level);
          if (own && col % kLevelD == 0)
            g.de[(int64_t)m * (g.Np / kLevelD) + n / kLevelD] = (uint8_t)level;
        }
        T4 dgv, duv;
#pragma unroll
        for (int j = 0; j < 4; ++j) dgv[j] = (T)(vg[j] * k), duv[j] = (T)(vu[j] * k);
        if (own) {
          T* o = dd + (int64_t)m * (2 * g.Np) + n;
          *reinterpret_cast<T4*>(o) = dgv;
          *reinterpret_cast<T4*>(o + g.Np) = duv;
        }
      }
      if (g.dt == nullptr) return;
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const float a = sa[row_of(p)];
        const bool ok = m0 + row_of(p) < g.M;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          dg[p][j] = ok && j < nn ? dg[p][j] * a : 0.f;
          du[p][j] = ok && j < nn ? du[p][j] * a : 0.f;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float kg = block_power(dg, j, levels[0][j], part), ku = block_power(du, j, levels[1][j], part);
#pragma unroll
        for (int p = 0; p < PASSES; p += 2) {
          // two neighbouring rows at once: they go to LDS in pairs
          typedef T T2 __attribute__((ext_vector_type(2)));
          const int r = 16 * part + row_of(p);  // even
          const int c0 = col + j, c1 = COLS + col + j;
          ttw[c0 * 32 + 4 * ((r >> 3) ^ ((c0 >> 2) & 7)) + ((r & 7) >> 1)] =
              __builtin_bit_cast(uint32_t, (T2{(T)(dg[p][j] * kg), (T)(dg[p + 1][j] * kg)}));
          ttw[c1 * 32 + 4 * ((r >> 3) ^ ((c1 >> 2) & 7)) + ((r & 7) >> 1)] =
              __builtin_bit_cast(uint32_t, (T2{(T)(du[p][j] * ku), (T)(du[p + 1][j] * ku)}));
        }
      }
      if (part == 3 && m0 < g.Mp) {
        if constexpr (DT == XF16) {
          if (lane < LPR) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (j >= nn) continue;
              uint32_t* o = reinterpret_cast<uint32_t*>(g.dte + (int64_t)(n + j) * (g.Mp / kLevelT) + (m0 - 48) / kLevelT);
              o[0] = levels[0][j];
              o[g.Nr * (g.Mp / kLevelT) / 4] = levels[1][j];
            }
          }
        }
        // whole 128-byte lines: 8 lanes on a column's 64 rows
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        T* dt = static_cast<T*>(g.dt);
#pragma unroll 4
        for (int it = 0; it < 2 * COLS / 8; ++it) {
          const int c = 8 * it + lane / 8, cn = n0 + c % COLS;
          if (cn >= g.N) continue;
          const u32x4_t x = *reinterpret_cast<const u32x4_t*>(ttw + c * 32 + 4 * ((lane & 7) ^ ((c >> 2) & 7)));
          T* o = dt + ((int64_t)(c / COLS) * g.Nr + cn) * g.Mp + (m0 - 48) + 8 * (lane & 7);
          *reinterpret_cast<u32x4_t*>(o) = x;
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      }
    }
  }
};

// The workgroup's row scales (plain, fp16: row factors) to LDS (0 for rows past M).
template <int EPI, int DT>
__device__ __forceinline__ void row_scales(const TileArgs& g, float* sa, int m0, int rows) {
  if constexpr (EPI == EPI_PARTIAL || (EPI == EPI_PLAIN && DT != XF16)) return;
  for (int i = threadIdx.x; i < rows; i += 256) sa[i] = m0 + i < g.M ? g.sa[m0 + i] : 0.f;
}

// Tile of work item b of n_tiles x m_tiles: consecutive items on one XCD (the
// dispatcher deals workgroups round-robin over the 8), and among them GM row
// tiles of a column tile before the next column, so that the workgroups of an
// XCD that run together share rows and columns through its L2.
__device__ __forceinline__ void tile_of(int b, int n_tiles, int m_tiles, int* mt, int* nt) {
  constexpr int GM = 4;
  const int total = n_tiles * m_tiles, q = total / 8, r = total % 8, x = b % 8;
  const int w = x * q + min(x, r) + b / 8;
  const int per = GM * n_tiles, g = w / per, i = w % per;
  const int gm = min(GM, m_tiles - g * GM);
  *mt = g * GM + i % gm;
  *nt = i / gm;
}

}  // namespace qmm
