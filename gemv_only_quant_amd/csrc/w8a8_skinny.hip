// w8a8_skinny.hip -- int8 x int8 products of a decode batch (5 to 64 tokens,
// plain and gated) on v_mfma_i32_16x16x64_i8: bound by reading the weights.
//
// A workgroup owns all tokens (MT 16-row tiles) and NT strips of 16 columns; its
// waves split K in turns of 256 bytes, so that rows whose stride is a power of two
// spread over the L2's channels, and add their whole sums in LDS at the end
// (integers: any order gives the same).  A wave's weights and codes come in items
// of 128 bytes of every row, by loads straight to its own part of LDS, D items in
// flight, and are read from there as operands: no barrier before the end.
//   Why through LDS: operands as the matrix cores want them have neighbouring
// lanes in different rows, and the address units then take a load's 64 lanes one
// by one (64 rows x 4096 x 14336: 22.8 us, bound by that); 8 lanes on a 128-byte
// line take a quarter of the time.
#include <type_traits>

#include "w8a8_tile.h"

namespace qmm {

// LDS of a workgroup: the waves' rings; in their place at the end the sums; then
// the scales of the tokens and of the strips' columns.
// Four waves with at most four items each are enough to keep a CU's loads busy (codes, us:
// 16 rows x 14336 x 1024 11.0, with 8 waves 11.6, with 8 items 12.6; 8 x 8192 x 8192
// 14.1 / 16.1 / 16.5).
constexpr int kSkinnyLds = 144 << 10;
constexpr int kSkinnyWaves = 4;
template <int MT, int NT> struct SkinnyPlan {
  static constexpr int WV = kSkinnyWaves;
  static constexpr int ITEM = (MT + NT) * 2048;  // bytes
  static constexpr int FIT = kSkinnyLds / (WV * ITEM);
  static constexpr int D = FIT < 2 ? 2 : (FIT > 4 ? 4 : FIT);
  static constexpr int LD = 16 * NT + 4;  // row of the sums
  static constexpr int RING = WV * D * ITEM, SUMS = 16 * MT * LD * 4;
  static constexpr int BYTES = (RING > SUMS ? RING : SUMS) + (16 * MT + 16 * NT) * 4;
  static_assert(BYTES <= 160 << 10, "LDS of a CU");
};

// (a device function beside its kernel: the host pass drops a kernel whose own
// body has loads straight to LDS)
template <int MT, int NT, bool GATED>
__device__ __forceinline__ void skinny_body(const TileArgs& g, u32x4_t* lds) {
  typedef SkinnyPlan<MT, NT> P;
  constexpr int COLS = GATED ? 8 * NT : 16 * NT;  // output columns of the workgroup
  constexpr int WV = kSkinnyWaves, LD = P::LD, D = P::D, UNITS = 2 * (MT + NT);
  int* sums = reinterpret_cast<int*>(lds);
  float* scales = reinterpret_cast<float*>(lds) + (P::RING > P::SUMS ? P::RING : P::SUMS) / 4;
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
  buf_t rows[MT + NT];
#pragma unroll
  for (int s = 0; s < NT; ++s)
    rows[s] = GATED ? rows_of(g.b[s / (NT / 2)], g.ldb, n0 + 16 * (s % (NT / 2)), g.N)
                    : rows_of(g.b[0], g.ldb, n0 + 16 * s, g.N);
#pragma unroll
  for (int i = 0; i < MT; ++i) rows[NT + i] = rows_of(g.a, g.lda, 16 * i, g.M);

  // Item i of this wave: 128 bytes of K from byte k_of(i) on.  A load (1 KiB) is 8
  // rows of a strip; chunk c of row r lies at slot 8 r + (c ^ (r / 2 % 8)), so lane
  // p of the strip's half h fetches chunk (p % 8) ^ (r / 2 % 8) of row r = 8 h + p /
  // 8.  Past the end the offset lies outside every buffer: nothing is read.
  auto k_of = [&](int i) { return (wave + WV * (i >> 1)) * 256 + 128 * (i & 1); };
  int ao[2], bo[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int chunk = 16 * ((lane & 7) ^ ((4 * h + (lane >> 4)) & 7));
    ao[h] = (8 * h + (lane >> 3)) * lda + chunk;
    bo[h] = (8 * h + (lane >> 3)) * ldb + chunk;
  }
  u32x4_t* ring = lds + wave * (P::RING / WV / 16);
  auto load = [&](int i, int slot) {
    const int k = k_of(i), at = k < kb ? k : 0x60000000;
    auto to = [&](int u) {
      return (__attribute__((address_space(3))) void*)(ring + slot * (P::ITEM / 16) + 64 * u);
    };
#pragma unroll
    for (int u = 0; u < 2 * NT; ++u)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rows[u / 2], to(u), 16, bo[u % 2] + at, 0, 0, kStream);
#pragma unroll
    for (int u = 2 * NT; u < UNITS; ++u)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rows[u / 2], to(u), 16, ao[u % 2] + at, 0, 0, 0);
  };
  // operand j (k step) of strip s of the item in `slot`
  const int swz = (l16 >> 1) & 7;
  auto frag = [&](int s, int j, int slot) {
    return ring[slot * (P::ITEM / 16) + 128 * s + 8 * l16 + ((4 * j + quad) ^ swz)];
  };
  i32x4_t acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int s = 0; s < NT; ++s) acc[i][s] = i32x4_t{0, 0, 0, 0};

  {
    const int i = threadIdx.x;
    if (i < 16 * MT) scales[i] = i < g.M ? g.sa[i] : 0.f;
    else if (i < 16 * MT + 16 * NT) {
      const int c = i - 16 * MT, n = n0 + c % COLS;
      scales[i] = n < g.N ? g.sb[GATED ? c / COLS : 0][n] : 0.f;
    }
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int d = 0; d < D; ++d) load(d, d);

  // vmcnt(N) with the other counters at maximum
  constexpr int LEFT = (D - 1) * UNITS;
  static_assert(LEFT < 64, "loads in flight");
  constexpr int kWaitItem = (LEFT & 15) | ((LEFT >> 4) << 14) | 0x0F70;
  for (int i = 0; k_of(i) < kb; i += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      // (items past the end are read and multiplied as zeros: their operands of
      // A are cleared below)
      const int k = k_of(i + d);
      __builtin_amdgcn_s_waitcnt(kWaitItem);
      __builtin_amdgcn_sched_barrier(0);
      u32x4_t a[MT][2], b[NT][2];
#pragma unroll
      for (int s = 0; s < NT; ++s)
#pragma unroll
        for (int j = 0; j < 2; ++j) b[s][j] = frag(s, j, d);
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) a[t][j] = frag(NT + t, j, d);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot is free
      __builtin_amdgcn_sched_barrier(0);
      load(i + d + D, d);
      if (k + 128 > kb) {  // the codes' bytes past K (whatever B holds there meets zeros)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int j = 0; j < 2; ++j) a[t][j] = clear_tail(a[t][j], k + 64 * j + 16 * quad, kb);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int s = 0; s < NT; ++s) acc[t][s] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a[t][j]),
                                                              __builtin_bit_cast(i32x4_t, b[s][j]),
                                                              acc[t][s], 0, 0, 0);
    }
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): no load may land in the sums
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * MT * LD; i += 64 * WV) sums[i] = 0;
  __syncthreads();
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
    for (int i = threadIdx.x; i < 16 * MT * PER_ROW; i += 64 * WV) {
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

template <int MT, int NT, bool GATED>
__global__ __launch_bounds__(64 * kSkinnyWaves) void skinny_kernel(TileArgs g) {
  // one array for everything: with a second one in LDS the compiler waits for
  // all memory before it reads any
  __shared__ u32x4_t lds[(SkinnyPlan<MT, NT>::BYTES + 15) / 16];
  skinny_body<MT, NT, GATED>(g, lds);
}

// ---------------------------------------------------------------- host side
bool skinny_fits(int M) { return M <= 64; }

template <int MT, int NT, bool GATED>
static hipError_t launch_skinny_k(const TileArgs& t, hipStream_t s) {
  constexpr int COLS = GATED ? 8 * NT : 16 * NT;
  return launch_kernel(skinny_kernel<MT, NT, GATED>, dim3((unsigned)((t.N + COLS - 1) / COLS)),
                       dim3(64 * kSkinnyWaves), s, t);
}

// Strips per workgroup: 4 share each reading of the codes where that leaves at
// least 192 workgroups (codes, us, 4 / 2 / 1 strips: 64 rows x 4096 x 14336 17.9 /
// 24.5 / 34.2; 16 rows 14.9 / 16.8 / 17.0), else 2 with more than 16 rows, 1 with
// up to 16 (8 x 8192 x 8192 18.9 / 16.5 / 14.0, 16 x 14336 x 1024 24.5 / 15.1 / 10.9)
// or where 2 leave too few.  A pair of products has at least one strip of each.
template <int MT, bool GATED>
static hipError_t launch_skinny_m(const TileArgs& t, hipStream_t s) {
  constexpr int W = GATED ? 8 : 16;
  if (t.N / (4 * W) >= 192) return launch_skinny_k<MT, 4, GATED>(t, s);
  if (GATED || (MT > 1 && t.N / (2 * W) >= 192)) return launch_skinny_k<MT, 2, GATED>(t, s);
  if constexpr (!GATED) return launch_skinny_k<MT, 1, GATED>(t, s);
  return hipErrorInvalidValue;
}

hipError_t launch_skinny(const TileArgs& t, bool gated, hipStream_t s) {
  if (t.M <= 16) return gated ? launch_skinny_m<1, true>(t, s) : launch_skinny_m<1, false>(t, s);
  if (t.M <= 32) return gated ? launch_skinny_m<2, true>(t, s) : launch_skinny_m<2, false>(t, s);
  return gated ? launch_skinny_m<4, true>(t, s) : launch_skinny_m<4, false>(t, s);
}

}  // namespace qmm
