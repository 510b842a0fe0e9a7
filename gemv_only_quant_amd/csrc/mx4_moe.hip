// mx4_moe.hip -- a mixture-of-experts layer for up to 64 tokens, experts' weights
// in packed microscaled 4-bit codes, activations as they are.
//
//   h[t][j] = w[t][j] act(Wg_e x[t]) * (Wu_e x[t]),  y[t] = sum_j Wd_e h[t][j]
//
// Bound by reading the weights of the experts that some token chose, once.  The
// products run on the 16-bit matrix cores: a code times its scale is exact in
// bf16, whose exponents reach as far as the scales', and an activation of more
// bits is a sum of bf16 parts (fp16: 2, fp32: 3, exact), each multiplied in turn;
// in the weights' shadow that costs nothing.  Rows of the product are the tokens
// themselves, zeros where a token did not choose the expert: so the second half
// adds all experts in its accumulators.
#include "mx4_device.h"

namespace qmm {

// The workgroup's view of the routing: tokens' ids and weights in LDS, and the
// experts that some token chose, ascending.
struct MoeRouting {
  int ids[kMoeTokens * kMoeTopK];
  float w[kMoeTokens * kMoeTopK];
  int list[kMoeExperts];
  int flag[kMoeExperts];
  int count;
};

__device__ __forceinline__ void load_routing(MoeRouting& r, const int* ids, const float* w, int T, int k, int E) {
  const int tid = threadIdx.x, n = blockDim.x;
  for (int i = tid; i < E; i += n) r.flag[i] = 0;
  __syncthreads();
  for (int i = tid; i < T * k; i += n) {
    const int e = ids[i];
    r.ids[i] = e;
    r.w[i] = w[i];
    if (e >= 0) r.flag[e] = 1;
  }
  __syncthreads();
  if (tid < 64) {
    int c = 0;
    for (int b = 0; b < E; b += 64) {
      const bool on = b + tid < E && r.flag[b + tid] != 0;
      const uint64_t m = __ballot(on);
      if (on) r.list[c + __popcll(m & ((uint64_t(1) << tid) - 1))] = b + tid;
      c += __popcll(m);
    }
    if (tid == 0) r.count = c;
  }
  __syncthreads();
}

// Whether token `t` chose expert e: the first of its places that holds it, or -1;
// and the sum of all such places' weights.
__device__ __forceinline__ int place_of(const MoeRouting& r, int t, int T, int k, int e, float* w) {
  int at = -1;
  float sum = 0.f;
  if (t < T)
    for (int j = 0; j < k; ++j)
      if (r.ids[t * k + j] == e) {
        at = at < 0 ? j : at;
        sum += r.w[t * k + j];
      }
  *w = sum;
  return at;
}

// v as a sum of N bf16 values, 8 bits of it each: all but the last cut off, so that
// none leaves the range, the last rounded (fp16 in 2 and fp32 in 3 parts are exact
// but for what lies below bf16's smallest value).  What is not finite is its first part
// alone.
template <int N> __device__ __forceinline__ void parts_of(float v, uint16_t (&p)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i == N - 1) {
      const __bf16 h = (__bf16)v;
      p[i] = __builtin_bit_cast(uint16_t, h);
    } else {
      uint32_t h = __builtin_bit_cast(uint32_t, v) & 0xFFFF0000u;
      if (v != v) h = 0x7FC00000u;
      p[i] = (uint16_t)(h >> 16);
      v = (h & 0x7F800000u) == 0x7F800000u ? 0.f : v - __builtin_bit_cast(float, h);
    }
  }
}

// ---- routing, and the activations as parts ------------------------------------
__device__ __forceinline__ float as_f32(const void* p, int64_t i, int dtype) {
  if (dtype == YF32) return static_cast<const float*>(p)[i];
  if (dtype == XF16) return (float)static_cast<const _Float16*>(p)[i];
  return (float)static_cast<const __bf16*>(p)[i];
}

// Order of logits as unsigned numbers: NaN above infinity, -infinity lowest (0 is below all).
__device__ __forceinline__ uint32_t order_of(float v) {
  if (v != v) return 0xFFFFFFFFu;
  v = v == 0.f ? 0.f : v;  // -0 equals 0
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

struct MoeBufs {
  int* ids;
  float* w;
  uint16_t* x;
  uint16_t* h;
};

template <int XP>
__global__ __launch_bounds__(256) void moe_route_kernel(MoeArgs g, MoeBufs o, int Dp) {
  const int t = (int)blockIdx.x, tid = threadIdx.x, lane = tid & 63, k = g.top_k;
  if (tid < 64) {
    if (g.logits == nullptr) {
      for (int j = lane; j < k; j += 64) {
        const int64_t i = (int64_t)t * k + j;
        const int64_t e = g.ids_size == 8 ? static_cast<const int64_t*>(g.ids)[i] : static_cast<const int32_t*>(g.ids)[i];
        o.ids[i] = e >= 0 && e < g.E ? (int)e : -1;
        o.w[i] = as_f32(g.weights, i, g.weights_dtype);
      }
    } else {
      // k times the largest key (order, then lowest index) that is below the last
      float first = 0.f, sum = 0.f, all = 0.f;
      uint64_t last = ~uint64_t(0);
      float mine = 0.f;
      int chosen = -1;
      for (int j = 0; j < k; ++j) {
        uint64_t best = 0;
        for (int e = lane; e < g.E; e += 64) {
          const float v = as_f32(g.logits, (int64_t)t * g.ldl + e, g.logits_dtype);
          if (v == -__builtin_inff()) continue;
          const uint64_t key = ((uint64_t)order_of(v) << 32) | (uint32_t)(kMoeExperts - e);
          if (key < last && key > best) best = key;
        }
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) {
          const uint64_t other = __shfl_xor((unsigned long long)best, d, 64);
          best = other > best ? other : best;
        }
        if (best == 0) break;  // no expert is left
        last = best;
        const int e = kMoeExperts - (int)(uint32_t)best;
        const float v = as_f32(g.logits, (int64_t)t * g.ldl + e, g.logits_dtype);
        if (j == 0) first = v;
        const float p = v <= first ? exp_f32(v - first) : __builtin_nanf("");
        sum += first - first == 0.f ? p : __builtin_nanf("");
        if (lane == j) mine = p, chosen = e;
      }
      if (!g.renormalize) {
        for (int e = lane; e < g.E; e += 64) {
          const float v = as_f32(g.logits, (int64_t)t * g.ldl + e, g.logits_dtype);
          if (v <= first) all += exp_f32(v - first);
        }
        const float s = wave_sum(all);
        sum = sum == sum ? s : sum;
      }
      if (lane < k) {
        o.ids[t * k + lane] = chosen;
        o.w[t * k + lane] = mine / sum;
      }
    }
  }
  for (int i = tid; i < Dp; i += 256) {
    uint16_t p[XP];
    parts_of<XP>(i < g.D ? as_f32(g.x, (int64_t)t * g.ldx + i, g.x_dtype) : 0.f, p);
#pragma unroll
    for (int q = 0; q < XP; ++q) o.x[((int64_t)q * g.T + t) * Dp + i] = p[q];
  }
}

// ---- first half ----------------------------------------------------------------
// A workgroup: 16 columns of h of one expert, the waves taking steps of K in turn.
constexpr int kUpWaves = 4;

template <int MT, int XP, int HP>
__global__ __launch_bounds__(64 * kUpWaves) void moe_up_kernel(MoeArgs g, MoeBufs o, int Dp, int Ip) {
  __shared__ MoeRouting r;
  __shared__ float sums[kUpWaves][2][16][17];
  load_routing(r, o.ids, o.w, g.T, g.top_k, g.E);
  const int slot = (int)blockIdx.y;
  if (slot >= r.count) return;
  const int e = r.list[slot];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, quad = lane >> 4;
  const int strip = (int)blockIdx.x;
  const int steps = 4 * mx4_chunks(g.D);
  const int64_t at = (int64_t)e * mx4_weight_bytes(g.I, g.D) + (int64_t)strip * mx4_strip_bytes(g.D);
  float wt;
  const int place = place_of(r, lane, g.T, g.top_k, e, &wt);
  const uint64_t members = __ballot(place >= 0);
  f32x4_t acc[MT][2];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i][0] = acc[i][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int s = wave; s < steps; s += kUpWaves) {
    u32x4_t c[2];
    float sc[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const uint8_t* w = (p == 0 ? g.wg : g.wu) + at + (int64_t)kChunkBytes * (s / 4);
      c[p] = *reinterpret_cast<const u32x4_t*>(w + 1024 * (s % 4) + 16 * lane);
      sc[p] = scale_f32(w[4096 + 4 * lane + s % 4]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bf16x8_t bg = __builtin_bit_cast(bf16x8_t, bf16_of_codes(c[0][i], sc[0]));
      const bf16x8_t bu = __builtin_bit_cast(bf16x8_t, bf16_of_codes(c[1][i], sc[1]));
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (((members >> (16 * m)) & 0xFFFF) == 0) continue;
        const int t = 16 * m + l16;
#pragma unroll
        for (int q = 0; q < XP; ++q) {
          u32x4_t a = {0u, 0u, 0u, 0u};
          if ((members >> t) & 1)
            a = *reinterpret_cast<const u32x4_t*>(o.x + ((int64_t)q * g.T + t) * Dp + 512 * (s / 4) + 32 * (4 * quad + s % 4) + 8 * i);
          const bf16x8_t av = __builtin_bit_cast(bf16x8_t, a);
          acc[m][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, bg, acc[m][0], 0, 0, 0);
          acc[m][1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, bu, acc[m][1], 0, 0, 0);
        }
      }
    }
  }
  for (int m = 0; m < MT; ++m) {
    if (((members >> (16 * m)) & 0xFFFF) == 0) continue;
    __syncthreads();
#pragma unroll
    for (int mm = 0; mm < MT; ++mm)
      if (mm == m) {
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int q = 0; q < 4; ++q) sums[wave][p][4 * quad + q][l16] = acc[mm][p][q];
      }
    __syncthreads();
    const int row = threadIdx.x / 16, col = threadIdx.x % 16, t = 16 * m + row;
    // what token t's lane knows
    const int at_t = __shfl(place, t & 63, 64);
    const float w_t = __shfl(wt, t & 63, 64);
    float gv = 0.f, uv = 0.f;
#pragma unroll
    for (int q = 0; q < kUpWaves; ++q) gv += sums[q][0][row][col], uv += sums[q][1][row][col];
    if (at_t >= 0) {
      float h = 0.f;
      with_act(g.act, [&](auto a) {
        float d;
        h = act_parts<decltype(a)::value>(gv, &d) * uv * w_t;
      });
      uint16_t p[HP];
      parts_of<HP>(h, p);
#pragma unroll
      for (int q = 0; q < HP; ++q)
        o.h[((int64_t)q * g.T * g.top_k + t * g.top_k + at_t) * Ip + 16 * strip + col] = p[q];
    }
  }
}

// ---- second half ---------------------------------------------------------------
// A workgroup: 16 columns of y, the waves taking steps of every chosen expert in turn.
constexpr int kDownWaves = 8;

template <int MT, int HP>
__global__ __launch_bounds__(64 * kDownWaves) void moe_down_kernel(MoeArgs g, MoeBufs o, int Ip) {
  __shared__ MoeRouting r;
  __shared__ float sums[kDownWaves][16][17];
  load_routing(r, o.ids, o.w, g.T, g.top_k, g.E);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, quad = lane >> 4;
  const int strip = (int)blockIdx.x;
  const int steps = 4 * mx4_chunks(g.I);
  f32x4_t acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int items = r.count * steps;
  int slot = -1, place = -1;
  uint64_t members = 0;
  const uint8_t* w = nullptr;
  for (int it = wave; it < items; it += kDownWaves) {
    const int s = it % steps;
    if (it / steps != slot) {
      slot = it / steps;
      const int e = r.list[slot];
      float wt;
      place = place_of(r, lane, g.T, g.top_k, e, &wt);
      members = __ballot(place >= 0);
      w = g.wd + (int64_t)e * mx4_weight_bytes(g.D, g.I) + (int64_t)strip * mx4_strip_bytes(g.I);
    }
    const uint8_t* wc = w + (int64_t)kChunkBytes * (s / 4);
    const u32x4_t c = *reinterpret_cast<const u32x4_t*>(wc + 1024 * (s % 4) + 16 * lane);
    const float sc = scale_f32(wc[4096 + 4 * lane + s % 4]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bf16x8_t b = __builtin_bit_cast(bf16x8_t, bf16_of_codes(c[i], sc));
      const int kk = 512 * (s / 4) + 32 * (4 * quad + s % 4) + 8 * i;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (((members >> (16 * m)) & 0xFFFF) == 0) continue;
        const int t = 16 * m + l16;
        const int at_t = __shfl(place, t, 64);
#pragma unroll
        for (int q = 0; q < HP; ++q) {
          u32x4_t a = {0u, 0u, 0u, 0u};
          if (at_t >= 0 && kk < Ip)
            a = *reinterpret_cast<const u32x4_t*>(o.h + ((int64_t)q * g.T * g.top_k + t * g.top_k + at_t) * Ip + kk);
          acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), b, acc[m], 0, 0, 0);
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q) sums[wave][4 * quad + q][l16] = acc[m][q];
    __syncthreads();
    const int row = threadIdx.x / 16, col = threadIdx.x % 16, t = 16 * m + row, n = 16 * strip + col;
    if (row < 16 && t < g.T && n < g.D) {
      float v = 0.f;
#pragma unroll
      for (int q = 0; q < kDownWaves; ++q) v += sums[q][row][col];
      with_y(g.y, g.y_dtype, [&](auto* yt) {
        typedef typename std::remove_pointer<decltype(yt)>::type Y;
        yt[(int64_t)t * g.ldy + n] = (Y)v;
      });
    }
  }
}

// ---------------------------------------------------------------- host side
MoePlan plan_moe(int T, int D, int I, int top_k, int x_dtype, int y_dtype) {
  MoePlan p{};
  p.xparts = x_dtype == YF32 ? 3 : x_dtype == XF16 ? 2 : 1;
  p.hparts = y_dtype == YF32 ? 3 : 2;
  p.Dp = (int)round_up(D, 512);
  p.Ip = (int)round_up(I, 16);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (size_t)round_up((int64_t)bytes, 256);
    return o;
  };
  p.ids = take((size_t)T * top_k * 4);
  p.w = take((size_t)T * top_k * 4);
  p.x = take((size_t)p.xparts * T * p.Dp * 2);
  p.h = take((size_t)p.hparts * T * top_k * p.Ip * 2);
  p.bytes = at;
  return p;
}

template <int MT, int XP, int HP>
static hipError_t moe_t(const MoeArgs& a, const MoePlan& p, const MoeBufs& o, hipStream_t s) {
  hipError_t e = launch_kernel(moe_route_kernel<XP>, dim3((unsigned)a.T), dim3(256), s, a, o, p.Dp);
  if (e != hipSuccess) return e;
  const int slots = a.T * a.top_k < a.E ? a.T * a.top_k : a.E;
  e = launch_kernel(moe_up_kernel<MT, XP, HP>, dim3((unsigned)((a.I + 15) / 16), (unsigned)slots),
                    dim3(64 * kUpWaves), s, a, o, p.Dp, p.Ip);
  if (e != hipSuccess) return e;
  return launch_kernel(moe_down_kernel<MT, HP>, dim3((unsigned)((a.D + 15) / 16)), dim3(64 * kDownWaves), s, a,
                       o, p.Ip);
}

template <int MT, int XP>
static hipError_t moe_h(const MoeArgs& a, const MoePlan& p, const MoeBufs& o, hipStream_t s) {
  return p.hparts == 3 ? moe_t<MT, XP, 3>(a, p, o, s) : moe_t<MT, XP, 2>(a, p, o, s);
}

template <int MT> static hipError_t moe_x(const MoeArgs& a, const MoePlan& p, const MoeBufs& o, hipStream_t s) {
  switch (p.xparts) {
    case 1: return moe_h<MT, 1>(a, p, o, s);
    case 2: return moe_h<MT, 2>(a, p, o, s);
  }
  return moe_h<MT, 3>(a, p, o, s);
}

hipError_t launch_mx4_moe(const MoeArgs& a, const MoePlan& p, hipStream_t s) {
  char* ws = static_cast<char*>(a.ws);
  const MoeBufs o{reinterpret_cast<int*>(ws + p.ids), reinterpret_cast<float*>(ws + p.w),
                  reinterpret_cast<uint16_t*>(ws + p.x), reinterpret_cast<uint16_t*>(ws + p.h)};
  if (a.T <= 16) return moe_x<1>(a, p, o, s);
  return a.T <= 32 ? moe_x<2>(a, p, o, s) : moe_x<4>(a, p, o, s);
}

}  // namespace qmm
