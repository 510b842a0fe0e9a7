// w8a8_rows.hip -- int8 x int8 products of a few tokens (decode), plain and
// gated: the weights are read once, everything else is in their shadow.
//
//   y[m][n] = sx[m] sw[n] sum_k xq[m][k] W[n][k];  h = act(g) u
//
// A workgroup of 16 waves holds the tokens' codes in LDS: copied, or made
// there from values (each workgroup quantizes the few rows itself: 2 K bytes
// from L2 and a maximum, while its first weights are on their way; a launch of
// its own would cost more than the whole product).  A wave then takes output
// columns in turn: 16 contiguous bytes of a weight row per lane, 1 KiB per
// step, U steps per batch, two batches in flight, multiplied with
// v_dot4_i32_i8.  Where the columns are too few to occupy the chip, S waves
// share a column, each on every S-th batch.  Sums are int32 and exact, so neither
// the order of K nor the number of waves shows in the result.
#include <type_traits>

#include "w8a8_device.h"

namespace qmm {

// Sum over the wave's 64 lanes, in every lane.
__device__ __forceinline__ int wave_sum_i32(int v) {
#define QMM_DPP_ADD(ctrl, mask) v += __builtin_amdgcn_update_dpp(0, v, ctrl, mask, 0xF, false)
  QMM_DPP_ADD(0xB1, 0xF);   // quad_perm [1,0,3,2]
  QMM_DPP_ADD(0x4E, 0xF);   // quad_perm [2,3,0,1]
  QMM_DPP_ADD(0x124, 0xF);  // row_ror:4
  QMM_DPP_ADD(0x128, 0xF);  // row_ror:8
  QMM_DPP_ADD(0x142, 0xA);  // row_bcast:15 into rows 1 and 3
  QMM_DPP_ADD(0x143, 0xC);  // row_bcast:31 into rows 2 and 3
#undef QMM_DPP_ADD
  return __builtin_amdgcn_readlane(v, 63);
}

constexpr int kRowsWaves = 16;

// The first 56 bytes of arguments (up to sw0) arrive in registers.  ldx in
// elements, `base` columns per workgroup and one more for the first `rem`
// workgroups; opts: bits 0-2 M, 4-5 the output's type, 6-7 the activation, bit 8
// whole 16-byte loads of x.
template <int XT, int MB, int U, int S, bool GATED>
__global__ __launch_bounds__(64 * kRowsWaves) void rows_kernel(
    const int8_t* __restrict__ w0, const int8_t* __restrict__ w1, const void* __restrict__ x,
    int ldw, int ldx, int K, int base, int rem, int opts, const float* __restrict__ sw0,
    const float* __restrict__ sw1, const float* __restrict__ sx, void* __restrict__ y,
    int64_t ldy) {
  constexpr int P = GATED ? 2 : 1;
  extern __shared__ __align__(16) unsigned char lds[];
  __shared__ uint32_t part[kRowsWaves];
  __shared__ float scale[MB];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int M = opts & 7, ydt = (opts >> 4) & 3, act = (opts >> 6) & 3;
  const int K16 = (K + 15) & ~15;
  const int LDK = (K16 + 1023) & ~1023;  // bytes of a token's codes in LDS, whole steps

  // ---- this workgroup's columns (an even share, so that no CU ends much
  // later than another) and the weights' batches: item (column, U steps of K)
  const int wg = (int)blockIdx.x;
  const int n_begin = wg * base + min(wg, rem);
  const int n_end = n_begin + base + (wg < rem ? 1 : 0);
  const int batches = (LDK / 1024 + U - 1) / U;
  struct Item {
    int n, bt;          // column, batch of K
    u32x4_t w[P][U];
    uint32_t s[P];      // the column's scales, loaded behind its weights
  };
  // No load is under a branch (the compiler would then wait for all of them
  // wherever it waits for one): an item that does not exist has empty buffers,
  // which read zeros without touching memory, as do bytes past a row's end.
  auto load = [&](Item& it, bool ok) {
    const int64_t n = ok ? it.n : 0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const buf_t b = make_buf((p == 0 ? w0 : w1) + n * ldw, ok ? (uint32_t)K16 : 0u);
#pragma unroll
      for (int u = 0; u < U; ++u)
        it.w[p][u] = buf_load128_stream(b, (it.bt * U + u) * 1024 + 16 * lane);
    }
#pragma unroll
    for (int p = 0; p < P; ++p)
      it.s[p] = buf_load32(make_buf((p == 0 ? sw0 : sw1) + n, ok ? 4u : 0u), 0);
  };
  // the item after one: the next of this wave's batches, of the same column or
  // the next
  auto after = [&](const Item& it, Item& to) {
    to.n = it.n;
    to.bt = it.bt + S;
    if (to.bt >= batches) {
      to.n += kRowsWaves / S;
      to.bt = wave % S;
    }
  };
  Item a, b;
  a.n = n_begin + wave / S;
  a.bt = wave % S;
  // Values are requested before the weights: loads return in order, so the
  // maximum and the codes are formed while the weights are on their way.
  constexpr bool QUANT = XT != kTypeI8;
  if constexpr (!QUANT) load(a, a.n < n_end);

  // ---- codes to LDS -------------------------------------------------------
  if constexpr (XT == kTypeI8) {
    const int8_t* xc = static_cast<const int8_t*>(x);
    for (int m = 0; m < MB; ++m)
      for (int k = 16 * threadIdx.x; k < LDK; k += 16 * 64 * kRowsWaves) {
        u32x4_t c = {0u, 0u, 0u, 0u};
        if (m < M && k < K)
          c = clear_tail(*reinterpret_cast<const u32x4_t*>(xc + (int64_t)m * ldx + k), k, K);
        *reinterpret_cast<u32x4_t*>(lds + m * LDK + k) = c;
      }
    if (threadIdx.x < MB) scale[threadIdx.x] = (int)threadIdx.x < M ? sx[threadIdx.x] : 0.f;
  } else {
    // 16 / MB waves per row; the first two vectors of a lane stay in
    // registers between the maximum and the codes
    typedef typename Elem<XT>::type T;
    constexpr int WPR = kRowsWaves / MB;
    constexpr int STEP = WPR * 64 * 8;
    const int m = wave / WPR, t = (wave % WPR) * 64 + lane;
    const int Km = m < M ? K : 0;
    const buf_t row = make_buf(static_cast<const T*>(x) + (int64_t)(m < M ? m : 0) * ldx,
                               (uint32_t)(Km * sizeof(T)));
    const bool vec = (opts >> 8) & 1;
    auto get = [&](int k) { return vec ? load8<XT, true>(row, k) : load8<XT, false>(row, k); };
    Raw8<XT> v[2] = {};
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (i * STEP + 512 * (wave % WPR) < Km) v[i] = get(i * STEP + 8 * t);
    __builtin_amdgcn_sched_barrier(0);
    load(a, a.n < n_end);
    __builtin_amdgcn_sched_barrier(0);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) top = top8<XT>(v[i], top);
    for (int k = 2 * STEP + 8 * t; k < Km; k += STEP) top = top8<XT>(get(k), top);
    top = wave_max_u32(top_f32<XT>(top));
    if (lane == 0) part[wave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      const uint32_t o = part[m * WPR + w];
      top = o > top ? o : top;
    }
    const RowScale c = row_scale(top);
    if (t == 0) scale[m] = c.s;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = i * STEP + 8 * t;
      if (k < LDK) *reinterpret_cast<u32x2_t*>(lds + m * LDK + k) = codes8<XT>(v[i], c);
    }
#pragma unroll 1
    for (int k = 2 * STEP + 8 * t; k < LDK; k += STEP)
      *reinterpret_cast<u32x2_t*>(lds + m * LDK + k) = codes8<XT>(get(k), c);
  }
  after(a, b);
  // Whether this wave has a second item; its loads go out before the barrier.
  // Either branch below holds the barrier and a use of the first item of its
  // own: after a join the compiler waits for what either branch has loaded
  // (4096 x 4096 from values 6.3 us, 5.0 with the branches apart).
  const bool more = b.n < n_end && (S == 1 || b.n == a.n);

  int acc[P][MB];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int m = 0; m < MB; ++m) acc[p][m] = 0;
  // lane m stores token m's result for column n, from its whole sums
  auto put = [&](int n, int s0, int s1, const uint32_t (&s)[P]) {
    if (lane >= M) return;
    const float sa = scale[lane];
    float r = (float)s0 * (sa * __builtin_bit_cast(float, (uint32_t)s[0]));
    if constexpr (GATED) {
      const float u = (float)s1 * (sa * __builtin_bit_cast(float, (uint32_t)s[P - 1]));
      with_act(act, [&](auto a) {
        float d;
        r = act_parts<decltype(a)::value>(r, &d) * u;
      });
    }
    with_y(y, ydt, [&](auto* yt) {
      typedef typename std::remove_pointer<decltype(yt)>::type Y;
      yt[(int64_t)lane * ldy + n] = (Y)r;
    });
  };
  // this wave's sums of a column, token m's in lane m; and clears them
  auto totals = [&](int (&s)[2]) {
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const int w = wave_sum_i32(acc[p][m]);
        s[p] = lane == m ? w : s[p];
        acc[p][m] = 0;
      }
  };
  // multiplies an item; stores its column where that was the last batch
  auto use = [&](const Item& it) {
    if (it.n >= n_end) return;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (it.bt * U + u) * 1024;
      if (!rows_step_exists<S>(k, u, LDK)) break;
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const u32x4_t c = *reinterpret_cast<const u32x4_t*>(lds + m * LDK + k + 16 * lane);
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[p][m] = __builtin_amdgcn_sdot4((int)c[j], (int)it.w[p][u][j], acc[p][m], false);
      }
    }
    if (S == 1 && it.bt + 1 >= batches) {
      int s[2] = {0, 0};
      totals(s);
      put(it.n, s[0], s[1], it.s);
    }
  };
  if (!more) {
    __syncthreads();
    use(a);
  } else if constexpr (S == 1) {
    load(b, true);
    __syncthreads();
    while (a.n < n_end) {
      use(a);
      after(b, a);
      load(a, a.n < n_end);
      use(b);
      after(a, b);
      load(b, b.n < n_end);
    }
  } else {
    const int n = a.n;
    load(b, true);
    __syncthreads();
    while (a.n == n) {
      use(a);
      if (b.n != n) break;
      after(b, a);
      load(a, a.n == n);
      use(b);
      after(a, b);
      load(b, b.n == n);
    }
  }
  if constexpr (S > 1) {
    // one column for each S waves; every wave comes to the barrier
    const int n = n_begin + wave / S;
    __shared__ int share[kRowsWaves][2][MB];
    int s[2] = {0, 0};
    totals(s);
    if (lane < MB) share[wave][0][lane] = s[0], share[wave][1][lane] = s[1];
    __syncthreads();
    if (wave % S == 0 && n < n_end && lane < MB) {
#pragma unroll
      for (int i = 1; i < S; ++i) s[0] += share[wave + i][0][lane], s[1] += share[wave + i][1][lane];
      uint32_t sc[P];
#pragma unroll
      for (int p = 0; p < P; ++p) sc[p] = buf_load32(make_buf((p == 0 ? sw0 : sw1) + n, 4u), 0);
      put(n, s[0], s[1], sc);
    }
  }
}

// ---------------------------------------------------------------- host side
// LDS a workgroup may use for the codes: two workgroups per CU.
constexpr int kRowsLds = 64 << 10;

static int rows_lds(int mb, int K) { return mb * (int)round_up(round_up(K, 16), 1024); }

static int rows_bucket(int M) { return M <= 1 ? 1 : M <= 2 ? 2 : 4; }

bool rows_fits(int M, int K) { return M <= 4 && K >= 512 && rows_lds(rows_bucket(M), K) <= kRowsLds; }

struct RowsArgs {
  const W8A8Args* a;
  const void* x;
  int64_t ldx;
  int opts;
};

template <int XT, int MB, int U, int S, bool GATED>
static hipError_t launch_rows_k(const RowsArgs& r) {
  const W8A8Args& a = *r.a;
  const int cpw = kRowsWaves / S;
  const int wgs = (a.N + cpw - 1) / cpw;
  // Workgroups that are resident at once: two per CU, one of the gated kernel,
  // whose two weights take the registers of both (gated 1 x 4096 x 11008: 256
  // workgroups 16.9 us, 512 18.3; plain 1 x 4096 x 14336: 256 13.7, 512 11.6).
  const int cap = GATED ? 256 : 512;
  const int grid = S > 1 || wgs < cap ? wgs : cap;
  // S > 1: whole rounds of cpw columns, one per workgroup
  const int base = S > 1 ? cpw : a.N / grid, rem = S > 1 ? 0 : a.N % grid;
  const int8_t *w0 = a.w[0], *w1 = a.w[1];
  const void* x = r.x;
  int ldw = (int)a.ldw, ldx = (int)r.ldx, K = a.K, b = base, m = rem, o = r.opts;
  const float *s0 = a.sw[0], *s1 = a.sw[1], *sx = a.sx;
  void* y = a.y;
  int64_t ldy = a.ldy;
  void* p[] = {&w0, &w1, &x, &ldw, &ldx, &K, &b, &m, &o, &s0, &s1, &sx, &y, &ldy};
  return hipLaunchKernel(reinterpret_cast<const void*>(rows_kernel<XT, MB, U, S, GATED>),
                         dim3((unsigned)grid), dim3(64 * kRowsWaves), p, (size_t)rows_lds(MB, a.K),
                         a.stream);
}

template <int XT, int MB, bool GATED>
static hipError_t launch_rows_m(const RowsArgs& r) {
  const int steps = (r.a->K + 1023) / 1024;
  const int cpw = kRowsWaves / 4;
  // 4 waves share a column where the weight is long and narrow (1 x 14336 x
  // 1024: 6.9 us against 9.1, 4096 x 1024 4.7 against 5.0, 8192 x 2048 7.3
  // either way, 14336 x 4096 16.5 against 13.5)
  const bool split = r.a->N <= 2048 && r.a->N % cpw == 0 && r.a->K >= 4 * r.a->N;
  if (split) return launch_rows_k<XT, MB, 2, 4, GATED>(r);
  if (steps >= 4) return launch_rows_k<XT, MB, 4, 1, GATED>(r);
  return steps >= 2 ? launch_rows_k<XT, MB, 2, 1, GATED>(r) : launch_rows_k<XT, MB, 1, 1, GATED>(r);
}

template <int XT>
static hipError_t launch_rows_t(const RowsArgs& r) {
  const bool g = r.a->gated;
  switch (rows_bucket(r.a->M)) {
    case 1: return g ? launch_rows_m<XT, 1, true>(r) : launch_rows_m<XT, 1, false>(r);
    case 2: return g ? launch_rows_m<XT, 2, true>(r) : launch_rows_m<XT, 2, false>(r);
  }
  return g ? launch_rows_m<XT, 4, true>(r) : launch_rows_m<XT, 4, false>(r);
}

hipError_t launch_rows(const W8A8Args& a, const void* x, int x_dtype, int64_t ldx) {
  const bool vec = x_dtype != kTypeI8 && vec8_ok(x, ldx, a.K, x_dtype == YF32 ? 4 : 2);
  const RowsArgs r{&a, x, ldx, a.M | (a.y_dtype << 4) | (a.act << 6) | (vec ? 256 : 0)};
  switch (x_dtype) {
    case kTypeI8: return launch_rows_t<kTypeI8>(r);
    case XF16: return launch_rows_t<XF16>(r);
    case XBF16: return launch_rows_t<XBF16>(r);
  }
  return launch_rows_t<YF32>(r);
}

}  // namespace qmm
