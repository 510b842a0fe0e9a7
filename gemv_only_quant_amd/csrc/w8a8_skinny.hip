// w8a8_skinny.hip -- int8 x int8 products of a decode batch (5 to 64 tokens,
// plain and gated) on v_mfma_i32_16x16x64_i8: bound by reading the weights.
//
// A workgroup of 8 waves owns all tokens (MT 16-row tiles) and NT strips of 16
// columns; its waves split K in turns of 256 bytes, so that rows whose stride
// is a power of two spread over the L2's channels, and add their whole sums in
// LDS at the end (integers: any order gives the same).  Weights and codes go
// from memory straight into operands, 128 bytes of each row at a time (whole
// cache lines), two such items in flight; the codes are read again by every
// workgroup, from L2, NT strips per reading.  No barrier before the end.
#include <type_traits>

#include "w8a8_tile.h"

namespace qmm {

constexpr int kSkinnyWaves = 8;

template <int MT, int NT, bool GATED>
__global__ __launch_bounds__(64 * kSkinnyWaves) void skinny_kernel(TileArgs g) {
  constexpr int COLS = GATED ? 8 * NT : 16 * NT;  // output columns of the workgroup
  constexpr int LD = 16 * NT + 4;                 // row of the sums in LDS
  __shared__ int sums[16 * MT * LD];
  __shared__ float scales[16 * MT + 16 * NT];  // of the tokens, then of the strips' columns
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, quad = lane >> 4;
  const int n0 = (int)blockIdx.x * COLS;
  const int kb = g.kb, kb16 = (kb + 15) & ~15;
  const int lda = (int)g.lda, ldb = (int)g.ldb;

  // a buffer per 16 rows of either operand, that ends with its last row
  auto rows_of = [&](const void* p, int64_t ld, int first, int limit) {
    const int n = min(16, limit - first);
    return make_buf(static_cast<const char*>(p) + (int64_t)(n > 0 ? first : 0) * ld,
                    n > 0 ? (uint32_t)((n - 1) * (int)ld + kb16) : 0u);
  };
  buf_t ar[MT], br[NT];
#pragma unroll
  for (int i = 0; i < MT; ++i) ar[i] = rows_of(g.a, g.lda, 16 * i, g.M);
#pragma unroll
  for (int s = 0; s < NT; ++s)
    br[s] = GATED ? rows_of(g.b[s / (NT / 2)], g.ldb, n0 + 16 * (s % (NT / 2)), g.N)
                  : rows_of(g.b[0], g.ldb, n0 + 16 * s, g.N);
  // whole 128-byte lines of 8 rows per load (line_operands)
  const int ao = (l16 & 7) * lda + 16 * (quad + 4 * (l16 >> 3));
  const int bo = (l16 & 7) * ldb + 16 * (quad + 4 * (l16 >> 3));

  // item i of this wave: 128 bytes of K from byte k_of(i) on; past the end its
  // offset lies outside every buffer, which reads zeros and no memory
  struct Item {
    u32x4_t a[MT][2], b[NT][2];
  };
  auto k_of = [&](int i) { return (wave + kSkinnyWaves * (i >> 1)) * 256 + 128 * (i & 1); };
  auto load = [&](int i, Item& it) {
    const int k = k_of(i), at = k < kb ? k : 0x60000000;
    const int av = ao + at, bv = bo + at;
#pragma unroll
    for (int s = 0; s < NT; ++s)
#pragma unroll
      for (int j = 0; j < 2; ++j) it.b[s][j] = buf_load128_stream(br[s], bv + 8 * j * ldb);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) it.a[t][j] = buf_load128(ar[t], av + 8 * j * lda);
  };
  i32x4_t acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int s = 0; s < NT; ++s) acc[i][s] = i32x4_t{0, 0, 0, 0};
  auto use = [&](int i, Item& it) {
    const int k = k_of(i);
#pragma unroll
    for (int s = 0; s < NT; ++s) line_operands(it.b[s]);
#pragma unroll
    for (int t = 0; t < MT; ++t) line_operands(it.a[t]);
    if (k + 128 > kb) {  // the codes' bytes past K (whatever B holds there meets zeros)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) it.a[t][j] = clear_tail(it.a[t][j], k + 64 * j + 16 * quad, kb);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int s = 0; s < NT; ++s) acc[t][s] = mfma_t<kTypeI8>(it.a[t][j], it.b[s][j], acc[t][s]);
  };

  Item x, y;
  load(0, x);
  load(1, y);
  for (int i = threadIdx.x; i < 16 * MT * LD; i += 64 * kSkinnyWaves) sums[i] = 0;
  {
    const int i = threadIdx.x;
    if (i < 16 * MT) scales[i] = i < g.M ? g.sa[i] : 0.f;
    else if (i < 16 * MT + 16 * NT) {
      const int c = i - 16 * MT, n = n0 + c % COLS;
      scales[i] = n < g.N ? g.sb[GATED ? c / COLS : 0][n] : 0.f;
    }
  }
  __syncthreads();
  for (int i = 0; k_of(i) < kb; i += 2) {
    use(i, x);
    load(i + 2, x);
    use(i + 1, y);
    load(i + 3, y);
  }
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int s = 0; s < NT; ++s)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        __hip_atomic_fetch_add(&sums[(16 * t + 4 * quad + r) * LD + 16 * s + l16], acc[t][s][r],
                               __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
  __syncthreads();

  // 4 columns of a row per thread
  constexpr int PER_ROW = COLS / 4;
  with_y(g.y, g.y_dtype, [&](auto* yt) {
    typedef typename std::remove_pointer<decltype(yt)>::type Y;
    const bool vec = vec4_ok(yt, g.ldy, (int)sizeof(Y));
    for (int i = threadIdx.x; i < 16 * MT * PER_ROW; i += 64 * kSkinnyWaves) {
      const int m = i / PER_ROW, col = 4 * (i % PER_ROW), n = n0 + col;
      const int nn = min(4, g.N - n);
      if (m >= g.M || nn <= 0) continue;
      const float a = scales[m];
      const float* sc = scales + 16 * MT + col;
      const int* c = &sums[m * LD + col];
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = (float)c[j] * (a * sc[j]);
      }
      if constexpr (GATED)
        with_act(g.act, [&](auto act) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float d;
            v[j] = act_parts<decltype(act)::value>(v[j], &d) * ((float)c[COLS + j] * (a * sc[COLS + j]));
          }
        });
      store4(yt + (int64_t)m * g.ldy + n, v, nn, vec);
    }
  });
}

// ---------------------------------------------------------------- host side
bool skinny_fits(int M) { return M <= 64; }

template <int MT, int NT, bool GATED>
static hipError_t launch_skinny_k(const TileArgs& t, hipStream_t s) {
  constexpr int COLS = GATED ? 8 * NT : 16 * NT;
  return launch_kernel(skinny_kernel<MT, NT, GATED>, dim3((unsigned)((t.N + COLS - 1) / COLS)),
                       dim3(64 * kSkinnyWaves), s, t);
}

template <int MT, bool GATED>
static hipError_t launch_skinny_m(const TileArgs& t, hipStream_t s) {
  // strips per workgroup: more share each reading of the codes, fewer make
  // more workgroups
  static const int want = env_int("QMM_SKINNY8_NT");
  constexpr int W = GATED ? 8 : 16;
  int nt = 4;
  while (nt > (GATED ? 2 : 1) && t.N / (W * nt) < 192) nt /= 2;
  if (want > 0) nt = want;
  if (nt == 4) return launch_skinny_k<MT, 4, GATED>(t, s);
  if (nt == 2 || GATED) return launch_skinny_k<MT, 2, GATED>(t, s);
  if constexpr (!GATED) return launch_skinny_k<MT, 1, GATED>(t, s);
  return hipErrorInvalidValue;
}

hipError_t launch_skinny(const TileArgs& t, bool gated, hipStream_t s) {
  if (t.M <= 16) return gated ? launch_skinny_m<1, true>(t, s) : launch_skinny_m<1, false>(t, s);
  if (t.M <= 32) return gated ? launch_skinny_m<2, true>(t, s) : launch_skinny_m<2, false>(t, s);
  return gated ? launch_skinny_m<4, true>(t, s) : launch_skinny_m<4, false>(t, s);
}

}  // namespace qmm
