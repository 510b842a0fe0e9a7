// mx4_skinny.hip -- products of microscaled 4-bit codes for few rows, y = x^ W^t:
// bound by reading the weights once.  The packed strip is the matrix cores' operand:
// waves stream chunks of 512 values from memory straight to registers and multiply
// them by v_mfma_scale_f32_16x16x128_f8f6f4, a few instructions for each KiB; what the
// kernels differ in is where the activations' operand comes from.
//
//  rows    (few values) x is quantized by every workgroup itself, into LDS in the
//          operand's order, while its first weights are on their way: one launch;
//  packed  x comes packed as weights are, and is read as they are, in blocks of up to 64 rows.
//
// The waves of a workgroup split K (chunks in turn) and add their sums in LDS in a fixed order.
// us from one launch to the next, bf16: 1 x 4096 x 4096 3.7 (2.4 TB/s); 64 x 4096 x 14336 13.4 with x packed (2.5 TB/s), of
// which the product is 10.9: 224 workgroups read 140 KB of weights and as much of x each, all of it requested at once.
#include <type_traits>

#include "mx4_device.h"

namespace qmm {

// A chunk of a packed strip: a lane's 4 blocks and their scales.
struct Chunk {
  u32x4_t c[4];
  uint32_t s;
};
// (p NULL: zeros)
template <int AUX> __device__ __forceinline__ void load_chunk(Chunk& w, const uint8_t* p, int lane) {
  const buf_t b = make_buf(p, p != nullptr ? kChunkBytes : 0);
#pragma unroll
  for (int j = 0; j < 4; ++j) w.c[j] = __builtin_amdgcn_raw_buffer_load_b128(b, 16 * lane, 1024 * j, AUX);
  w.s = __builtin_amdgcn_raw_buffer_load_b32(b, 4096 + 4 * lane, 0, AUX);
}

// c += A B^t over 128 values of 16 rows each, both operands mx4: lane L holds block L / 16 (32 codes, 16 bytes) of
// row L % 16, and in byte J of its scale word that block's scale; the matrix cores apply the scales (255 gives NaN, 0 is
// 2^-127).  Products within a block are summed exactly; block sums and accumulator are aligned to the largest of them, and
// what falls below its last bits is dropped.
template <int J>
__device__ __forceinline__ f32x4_t mfma_block(const u32x4_t& a, const u32x4_t& b, const f32x4_t& c, uint32_t sa, uint32_t sb) {
  const i32x8_t x = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8_t y = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, J, (int)sa, J, (int)sb);
}

// ---- rows ------------------------------------------------------------------------
// LDS: x's codes, 16 bytes for each (chunk, j, q, row) of a block 4 q + j, then its scales, a
// word for each (chunk, q, row), then the waves' sums of two strips in turn.
__host__ __device__ constexpr int rows_code_bytes(int M, int chunks) { return chunks * M * 256; }
__host__ __device__ constexpr int rows_x_bytes(int M, int chunks) { return chunks * M * 272; }

// VEC: whole 16-byte loads of x; `opts`: bits 0-4 M, 5-6 the output's type
template <int XT, int KW, bool VEC>
__global__ __launch_bounds__(64 * KW) void mx4_rows_kernel(const uint8_t* __restrict__ w, const void* __restrict__ x,
                                                           int64_t ldx, int N, int K, int opts, int groups,
                                                           void* __restrict__ y, int64_t ldy) {
  typedef typename Elem<XT>::type T;
  extern __shared__ __align__(16) unsigned char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, quad = lane >> 4;
  const int M = opts & 31, ydt = (opts >> 5) & 3;
  const int chunks = mx4_chunks(K), strips = (N + 15) / 16;
  float* sums = reinterpret_cast<float*>(lds + rows_x_bytes(M, chunks));

  // ---- this wave's chunks of the workgroup's strips, a ring of them on its way
  constexpr int RING = 3;
  Chunk ring[RING];
  const int64_t strip_bytes = mx4_strip_bytes(K);
  int ls = (int)blockIdx.x, lc = wave;  // what is requested next
  auto request = [&](Chunk& c) {
    load_chunk<kStream>(c, ls < strips && lc < chunks ? w + ls * strip_bytes + (int64_t)kChunkBytes * lc : nullptr, lane);
    lc += KW;
    if (lc >= chunks) lc = wave, ls += groups;
  };

  // ---- x to LDS: a turn of a wave is a chunk of a row, 8 values a lane
  const int turns = M * chunks;
  auto get = [&](int t) {
    const int r = t / chunks, k = 512 * (t - r * chunks) + 8 * lane;
    return take8<XT, VEC>(static_cast<const T*>(x) + (int64_t)r * ldx, k, K);
  };
  // lane: quarter lane % 4 of block lane / 4 = 4 q + j
  const int pq = lane >> 4, pj = (lane >> 2) & 3;
  auto put = [&](int t, Raw8<XT>& v) {
    const int r = t / chunks, c = t - r * chunks;
    settle8<XT, VEC>(v, 512 * c + 8 * lane, K);
    uint32_t top = top_f32<XT>(top8<XT>(v, 0u));
    uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xF, 0xF, false);
    top = o > top ? o : top;
    o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x4E, 0xF, 0xF, false);
    top = o > top ? o : top;
    const uint32_t e = scale_byte(top);
    float f[8];
    floats8<XT>(v, f);
    *reinterpret_cast<uint32_t*>(lds + ((16 * c + 4 * pj + pq) * M + r) * 16 + 4 * (lane & 3)) = codes_of8(f, e);
    if ((lane & 3) == 0) lds[rows_code_bytes(M, chunks) + ((4 * c + pq) * M + r) * 4 + pj] = (uint8_t)e;
  };
  // loads return in order: all of x but each wave's last few turns goes first, then these turns'
  // values, then the weights, so that they are quantized while the weights are on their way
  constexpr int HELD = XT == YF32 ? 2 : 4;
  Raw8<XT> held[HELD];
  int t = wave;
  for (; t + HELD * KW < turns; t += HELD * KW) {
#pragma unroll
    for (int i = 0; i < HELD; ++i) held[i] = get(t + i * KW);
#pragma unroll
    for (int i = 0; i < HELD; ++i) put(t + i * KW, held[i]);
  }
#pragma unroll
  for (int i = 0; i < HELD; ++i)
    if (t + i * KW < turns) held[i] = get(t + i * KW);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < RING; ++i) request(ring[i]);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < HELD; ++i)
    if (t + i * KW < turns) put(t + i * KW, held[i]);
  __syncthreads();

  // ---- products
  const int row = l16 < M ? l16 : 0;
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  int c = wave, parity = 0;
  auto use = [&](const Chunk& b) {
    const int cc = c < chunks ? c : 0;  // (a wave without a chunk has zeros for weights)
    const unsigned char* p = lds + ((16 * cc + quad) * M + row) * 16;
    const uint32_t sa = *reinterpret_cast<const uint32_t*>(lds + rows_code_bytes(M, chunks) + ((4 * cc + quad) * M + row) * 4);
    auto a = [&](int j) { return *reinterpret_cast<const u32x4_t*>(p + 64 * j * M); };
    acc = mfma_block<0>(a(0), b.c[0], acc, sa, b.s);
    acc = mfma_block<1>(a(1), b.c[1], acc, sa, b.s);
    acc = mfma_block<2>(a(2), b.c[2], acc, sa, b.s);
    acc = mfma_block<3>(a(3), b.c[3], acc, sa, b.s);
  };
  auto finish = [&](int strip) {
    float* s = sums + parity * (KW * M * 16);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (4 * quad + r < M) s[(wave * M + 4 * quad + r) * 16 + l16] = acc[r];
    acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
    __syncthreads();
    const int m = threadIdx.x / 16, n = 16 * strip + (int)threadIdx.x % 16;
    if (m < M && n < N) {
      float v = 0.f;
#pragma unroll
      for (int q = 0; q < KW; ++q) v += s[(q * M + m) * 16 + threadIdx.x % 16];
      with_y(y, ydt, [&](auto* yt) {
        typedef typename std::remove_pointer<decltype(yt)>::type Y;
        yt[(int64_t)m * ldy + n] = (Y)v;
      });
    }
    parity ^= 1;
  };
  for (int strip = (int)blockIdx.x; strip < strips;) {
#pragma unroll
    for (int i = 0; i < RING; ++i) {
      if (strip < strips) {
        use(ring[i]);
        request(ring[i]);
        c += KW;
        if (c >= chunks) {
          finish(strip);
          c = wave;
          strip += groups;
        }
      }
    }
  }
}

// ---- packed ----------------------------------------------------------------------
// A workgroup: 16 MT rows (MT strips of the packed x) and PS strips of columns.
template <int MT, int PS, int KW, class Y>
__global__ __launch_bounds__(64 * KW, 1) void mx4_packed_kernel(Mx4Args g) {
  const int m0 = 16 * MT * (int)blockIdx.y;
  __shared__ float sums[KW][PS][16 * MT][17];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, quad = lane >> 4;
  const int chunks = mx4_chunks(g.K), s0 = PS * (int)blockIdx.x;
  const int strips = (g.N + 15) / 16, mt = (g.M - m0 + 15) / 16;
  const int64_t strip_bytes = mx4_strip_bytes(g.K);
  const uint8_t* rows = g.a + m0 / 16 * strip_bytes;
  struct Stage {
    Chunk a[MT], b[PS];
  };
  auto request = [&](Stage& s, int c) {
    const int64_t at = (int64_t)kChunkBytes * c;
#pragma unroll
    for (int p = 0; p < PS; ++p)
      load_chunk<kStream>(s.b[p], c < chunks && s0 + p < strips ? g.w + (s0 + p) * strip_bytes + at : nullptr, lane);
#pragma unroll
    for (int i = 0; i < MT; ++i) load_chunk<0>(s.a[i], c < chunks && i < mt ? rows + i * strip_bytes + at : nullptr, lane);
  };
  f32x4_t acc[MT][PS];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int p = 0; p < PS; ++p) acc[i][p] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto use = [&](const Stage& s) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int p = 0; p < PS; ++p) {
        acc[i][p] = mfma_block<0>(s.a[i].c[0], s.b[p].c[0], acc[i][p], s.a[i].s, s.b[p].s);
        acc[i][p] = mfma_block<1>(s.a[i].c[1], s.b[p].c[1], acc[i][p], s.a[i].s, s.b[p].s);
        acc[i][p] = mfma_block<2>(s.a[i].c[2], s.b[p].c[2], acc[i][p], s.a[i].s, s.b[p].s);
        acc[i][p] = mfma_block<3>(s.a[i].c[3], s.b[p].c[3], acc[i][p], s.a[i].s, s.b[p].s);
      }
  };
  Stage st[2];
  request(st[0], wave);
  request(st[1], wave + KW);
  for (int c = wave; c < chunks; c += 2 * KW) {
    use(st[0]);
    request(st[0], c + 2 * KW);
    use(st[1]);
    request(st[1], c + 3 * KW);
  }
#pragma unroll
  for (int p = 0; p < PS; ++p)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) sums[wave][p][16 * i + 4 * quad + r][l16] = acc[i][p][r];
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * MT * 16 * PS; i += 64 * KW) {
    const int m = i / (16 * PS), col = i % (16 * PS), n = 16 * s0 + col;
    if (m0 + m >= g.M || n >= g.N) continue;
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < KW; ++q) v += sums[q][col / 16][m][col % 16];
    static_cast<Y*>(g.y)[(int64_t)(m0 + m) * g.ldy + n] = (Y)v;
  }
}

// ---------------------------------------------------------------- host side
constexpr int kRowsLds = 64 << 10;

static int rows_lds(int M, int K, int waves) { return rows_x_bytes(M, mx4_chunks(K)) + 2 * waves * M * 16 * 4; }
// Where strips are too few to occupy the chip, more waves share each.
static int rows_waves(int M, int N, int K) { return (N + 15) / 16 <= 128 && rows_lds(M, K, 16) <= kRowsLds ? 16 : 8; }

// Workgroups of 64 rows and PS strips, where these are all on the chip at once.
static int64_t row_blocks(int M, int N, int PS) { return (((int64_t)N + 16 * PS - 1) / (16 * PS)) * (((int64_t)M + 63) / 64); }
static bool at_once(int M, int N, int PS) { return row_blocks(M, N, PS) <= 256; }

// More rows too, if blocks of 64 with 4 strips are all on the chip at once: waves that split K end sooner than a few tiles of
// 128 x 128 that have all of it (K = 4096, us from codes: 128 x 4096 10.6, tiles 20.2; 256 x 4096 13.9, tiles 20.3; with 2
// rounds of blocks, 192 x 11008, 34, tiles 21).
bool mx4_skinny_fits(int M, int N) { return M <= 64 || at_once(M, N, 4); }

// Every workgroup quantizes all of x: up to 32 Ki values this costs less than a launch (4096 x 4096, us: 1 row
// 3.8, 4 5.0, 8 6.2, 16 9.1; packed first 7.8 to 8.5).
bool mx4_rows_fits(int M, int K) {
  return M <= 16 && (int64_t)M * K <= (1 << 15) && rows_lds(M, K, 8) <= kRowsLds;
}

template <int XT, int KW, bool VEC>
static hipError_t rows_k(const Mx4Args& a, const void* x, int64_t ldx, hipStream_t s) {
  const int strips = (a.N + 15) / 16, lds = rows_lds(a.M, a.K, KW);
  // workgroups that are on the chip at once
  const int most = KW == 16 ? 256 : 512;
  int groups = strips < most ? strips : most, N = a.N, K = a.K, opts = a.M | (a.y_dtype << 5);
  const uint8_t* w = a.w;
  void* y = a.y;
  int64_t ldy = a.ldy;
  void* p[] = {&w, &x, &ldx, &N, &K, &opts, &groups, &y, &ldy};
  return hipLaunchKernel(reinterpret_cast<const void*>(mx4_rows_kernel<XT, KW, VEC>), dim3((unsigned)groups), dim3(64 * KW), p,
                         (size_t)lds, s);
}
template <int XT> static hipError_t rows_t(const Mx4Args& a, const void* x, int64_t ldx, hipStream_t s) {
  const bool vec = vec8_ok(x, ldx, a.K, XT == YF32 ? 4 : 2) && a.K % 8 == 0;
  if (rows_waves(a.M, a.N, a.K) == 16) return vec ? rows_k<XT, 16, true>(a, x, ldx, s) : rows_k<XT, 16, false>(a, x, ldx, s);
  return vec ? rows_k<XT, 8, true>(a, x, ldx, s) : rows_k<XT, 8, false>(a, x, ldx, s);
}
hipError_t launch_mx4_rows(const Mx4Args& a, const void* x, int x_dtype, int64_t ldx, hipStream_t s) {
  switch (x_dtype) {
    case XF16: return rows_t<XF16>(a, x, ldx, s);
    case XBF16: return rows_t<XBF16>(a, x, ldx, s);
  }
  return rows_t<YF32>(a, x, ldx, s);
}

template <int MT, int PS, int KW> static hipError_t packed_y(const Mx4Args& a, hipStream_t s) {
  const int64_t strips = ((int64_t)a.N + 15) / 16, most = kMaxGroups * 256 / (64 * KW) * PS;  // of a launch
  hipError_t e = hipSuccess;
  for (int64_t f = 0; f < strips && e == hipSuccess; f += most) {
    Mx4Args g = a;
    g.w += f * mx4_strip_bytes(a.K);
    g.y = static_cast<char*>(a.y) + 16 * f * (a.y_dtype == YF32 ? 4 : 2);
    g.N = (int)(a.N - 16 * f < 16 * most ? a.N - 16 * f : 16 * most);
    const dim3 grid((unsigned)((((int64_t)g.N + 15) / 16 + PS - 1) / PS), (unsigned)((g.M + 16 * MT - 1) / (16 * MT)));
    const dim3 block(64 * KW);
    switch (a.y_dtype) {
      case XF16: e = launch_kernel(mx4_packed_kernel<MT, PS, KW, _Float16>, grid, block, s, g); break;
      case XBF16: e = launch_kernel(mx4_packed_kernel<MT, PS, KW, __bf16>, grid, block, s, g); break;
      default: e = launch_kernel(mx4_packed_kernel<MT, PS, KW, float>, grid, block, s, g);
    }
  }
  return e;
}
// Up to 32 rows.  Strips of a workgroup: 4, or 2, as long as most CUs have one; x is read again for each.  (K = 4096, us, 1, 2
// and 4 strips: 16 x 4096 8.5, 9.1, 9.4; 16 x 6144 11.9, 9.4, 9.7; 16 x 12288 16.0, 13.9, 10.7.)
template <int MT> static hipError_t packed_m(const Mx4Args& a, hipStream_t s) {
  const int strips = (a.N + 15) / 16;
  if (strips >= 4 * 192) return packed_y<MT, 4, 4>(a, s);
  if (strips >= 2 * 192) return packed_y<MT, 2, 8>(a, s);
  return packed_y<MT, 1, MT == 1 ? 16 : 8>(a, s);
}
// Blocks of 64 rows: 2 strips while they are all on the chip at once, else 4 (K = 4096, us, 2 and 4: 64 x 4096 10.1, 13.0; 64 x
// 6144 10.8, 13.4; 64 x 12288 16.8, 14.6; 1 strip 11.3, 17.5 and 24.4).
hipError_t launch_mx4_skinny(const Mx4Args& a, hipStream_t s) {
  if (a.M <= 16) return packed_m<1>(a, s);
  if (a.M <= 32) return packed_m<2>(a, s);
  return at_once(a.M, a.N, 2) ? packed_y<4, 2, 4>(a, s) : packed_y<4, 4, 4>(a, s);
}

}  // namespace qmm
