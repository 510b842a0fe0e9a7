// mx4_moe.hip -- a mixture-of-experts layer for up to 64 tokens, experts' weights
// in packed microscaled 4-bit codes, activations as they are.
//
//   h[t][j] = w[t][j] act(Wg_e x[t]) * (Wu_e x[t]),  y[t] = sum_j Wd_e h[t][j]
//
// Bound by reading the weights of the experts that some token chose, once.  The
// products run on the 16-bit matrix cores: a code times its scale is exact in
// bf16, whose exponents reach as far as the scales', and an activation of more
// bits is a sum of bf16 parts (fp16: 2, fp32: 3, exact), each multiplied in turn;
// in the weights' shadow that costs nothing.  Rows of the product are an expert's tokens.
//
// Three launches: the tokens' choices, and x as parts; the first half; the second.
#include "mx4_device.h"

namespace qmm {

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

__device__ __forceinline__ float value_of(uint32_t order) {
  if (order == 0xFFFFFFFFu) return __builtin_nanf("");
  return __builtin_bit_cast(float, order & 0x80000000u ? order & 0x7FFFFFFFu : ~order);
}

// What the first launch leaves for the others, in the workspace.
struct MoeBufs {
  int* slots;      // the experts that some token chose, ascending, then -1
  uint64_t* who;   // the tokens of each of them, a bit each
  uint2* place;    // (slot, token): the first of its places that holds the expert, and the sum of all
                   // such places' weights
  uint16_t* x;     // (parts, T, Dp)
  uint16_t* h;     // (parts, T top_k, Ip)
};

// Workgroup 0: the tokens' choices and the tables above.  The others: x as parts.
constexpr int kRouteWaves = 16;

template <int XP>
__global__ __launch_bounds__(64 * kRouteWaves) void moe_route_kernel(MoeArgs g, MoeBufs o, int Dp, int slots) {
  const int tid = threadIdx.x, lane = tid & 63, k = g.top_k;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (blockIdx.x > 0) {
    const int units = Dp / 8;
    for (int u = ((int)blockIdx.x - 1) * 64 * kRouteWaves + tid; u < g.T * units; u += ((int)gridDim.x - 1) * 64 * kRouteWaves) {
      const int t = u / units, i = 8 * (u - t * units);
      uint16_t p[8][XP];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        parts_of<XP>(i + j < g.D ? as_f32(g.x, (int64_t)t * g.ldx + i + j, g.x_dtype) : 0.f, p[j]);
#pragma unroll
      for (int q = 0; q < XP; ++q) {
        u32x4_t v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = p[2 * j][q] | ((uint32_t)p[2 * j + 1][q] << 16);
        *reinterpret_cast<u32x4_t*>(o.x + ((int64_t)q * g.T + t) * Dp + i) = v;
      }
    }
    return;
  }
  __shared__ int ids[kMoeTokens * kMoeTopK];
  __shared__ float ws[kMoeTokens * kMoeTopK];
  __shared__ int list[kMoeExperts];
  __shared__ int flag[kMoeExperts];
  __shared__ int count;
  for (int i = tid; i < g.E; i += 64 * kRouteWaves) flag[i] = 0;
  __syncthreads();
  if (g.logits == nullptr) {
    for (int i = tid; i < g.T * k; i += 64 * kRouteWaves) {
      const int64_t e = g.ids_size == 8 ? static_cast<const int64_t*>(g.ids)[i] : static_cast<const int32_t*>(g.ids)[i];
      const bool ok = e >= 0 && e < g.E;
      ids[i] = ok ? (int)e : -1;
      ws[i] = as_f32(g.weights, i, g.weights_dtype);
      if (ok) flag[(int)e] = 1;
    }
  } else {
    for (int t = wave; t < g.T; t += kRouteWaves) {
      // k times the largest key (order, then lowest index) that is below the last; the first
      // 128 experts' keys stay in registers
      constexpr int HELD = 2;
      auto key_of = [&](int e) -> uint64_t {
        if (e >= g.E) return 0;
        const float v = as_f32(g.logits, (int64_t)t * g.ldl + e, g.logits_dtype);
        return v == -__builtin_inff() ? 0 : ((uint64_t)order_of(v) << 32) | (uint32_t)(kMoeExperts - e);
      };
      uint64_t held[HELD];
#pragma unroll
      for (int i = 0; i < HELD; ++i) held[i] = key_of(64 * i + lane);
      float first = 0.f, sum = 0.f, mine = 0.f;
      uint64_t last = ~uint64_t(0);
      int chosen = -1;
      for (int j = 0; j < k; ++j) {
        uint64_t best = 0;
#pragma unroll
        for (int i = 0; i < HELD; ++i) best = held[i] < last && held[i] > best ? held[i] : best;
        for (int e = 64 * HELD + lane; e < g.E; e += 64) {
          const uint64_t key = key_of(e);
          best = key < last && key > best ? key : best;
        }
        // the largest order, and of its lanes the largest rest (the lowest index)
        const uint32_t hi = wave_max_u32((uint32_t)(best >> 32));
        const uint32_t lo = wave_max_u32((uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
        if (hi == 0) break;  // no expert is left
        last = ((uint64_t)hi << 32) | lo;
        const float v = value_of(hi);
        if (j == 0) first = v;
        // (NaN, and infinity less infinity: the whole row)
        const float p = first - first == 0.f ? exp_f32(v - first) : __builtin_nanf("");
        sum += p;
        if (lane == j) mine = p, chosen = kMoeExperts - (int)lo;
      }
      if (!g.renormalize) {
        float all = 0.f;
        for (int e = lane; e < g.E; e += 64) all += exp_f32(as_f32(g.logits, (int64_t)t * g.ldl + e, g.logits_dtype) - first);
        sum = sum == sum ? wave_sum(all) : sum;
      }
      if (lane < k) {
        ids[t * k + lane] = chosen;
        ws[t * k + lane] = mine / sum;
        if (chosen >= 0) flag[chosen] = 1;
      }
    }
  }
  __syncthreads();
  if (wave == 0) {
    int c = 0;
    for (int b = 0; b < g.E; b += 64) {
      const bool on = b + lane < g.E && flag[b + lane] != 0;
      const uint64_t m = __ballot(on);
      if (on) list[c + __popcll(m & ((uint64_t(1) << lane) - 1))] = b + lane;
      c += __popcll(m);
    }
    if (lane == 0) count = c;
  }
  __syncthreads();
  for (int s = wave; s < slots; s += kRouteWaves) {
    const int e = s < count ? list[s] : -1;
    int at = -1;
    float w = 0.f;
    if (lane < g.T && e >= 0)
      for (int j = 0; j < k; ++j)
        if (ids[lane * k + j] == e) {
          at = at < 0 ? j : at;
          w += ws[lane * k + j];
        }
    const uint64_t m = __ballot(at >= 0);
    if (lane == 0) o.slots[s] = e, o.who[s] = m;
    o.place[64 * s + lane] = uint2{(uint32_t)at, __builtin_bit_cast(uint32_t, w)};
  }
}

// ---- what both halves share ------------------------------------------------------
constexpr int kNowhere = 0x70000000;  // an offset outside every buffer: a load reads zeros

// A chunk of a packed strip as operands: a lane's 4 blocks and their scales.
struct MoeChunk {
  u32x4_t c[4];
  uint32_t s;
};
// From the buffer of a strip's chunk; of the `nb` blocks that exist in it.
__device__ __forceinline__ void load_chunk(MoeChunk& w, const uint8_t* p, int nb, int lane) {
  const buf_t b = make_buf(p, p != nullptr ? kChunkBytes : 0);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w.c[j] = buf_load128_stream(b, 4 * (lane >> 4) + j < nb ? 1024 * j + 16 * lane : kNowhere);
  w.s = __builtin_amdgcn_raw_buffer_load_b32(b, 4096 + 4 * lane, 0, kStream);
}

// Row r of the product is the r-th token of the expert; its rows of activations from `off` bytes on
// (kNowhere: no such row), blocks 4 (lane / 16) + j of a chunk.
template <int P> struct MoeRows {
  u32x4_t a[P][4];
  __device__ __forceinline__ void load(const buf_t (&b)[P], int off, int j, int nb, int lane) {
    const int at = 4 * (lane >> 4) + j < nb ? off + 256 * (lane >> 4) + 64 * j : kNowhere;
#pragma unroll
    for (int q = 0; q < P; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) a[q][i] = buf_load128(b[q], at + 16 * i);
  }
};
// Buffers of the parts of `rows` rows of `ld` bf16 values.
template <int P> __device__ __forceinline__ void part_buffers(buf_t (&b)[P], const uint16_t* p, int rows, int ld) {
#pragma unroll
  for (int q = 0; q < P; ++q) b[q] = make_buf(p + (int64_t)q * rows * ld, 2u * (uint32_t)rows * (uint32_t)ld);
}

template <int P>
__device__ __forceinline__ void multiply(f32x4_t& acc, const MoeRows<P>& r, const u32x4_t& c, float scale) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bf16x8_t b = __builtin_bit_cast(bf16x8_t, bf16_of_codes(c[i], scale));
#pragma unroll
    for (int q = 0; q < P; ++q)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, r.a[q][i]), b, acc, 0, 0, 0);
  }
}

// ---- first half ----------------------------------------------------------------
// A workgroup: 16 columns of h of one expert, the waves taking chunks of K in turn.
constexpr int kUpWaves = 4;

template <int XP, int HP>
__global__ __launch_bounds__(64 * kUpWaves) void moe_up_kernel(MoeArgs g, MoeBufs o, int Dp, int Ip) {
  __shared__ float sums[kUpWaves][2][16][17];
  __shared__ int tok[kMoeTokens];
  __shared__ uint2 place[kMoeTokens];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, quad = lane >> 4;
  const int strip = (int)blockIdx.x, slot = (int)blockIdx.y;
  const int e = o.slots[slot];
  const uint64_t who = o.who[slot];
  if (e < 0) return;
  const int chunks = mx4_chunks(g.D), blocks = mx4_blocks(g.D);
  const int64_t at = (int64_t)e * mx4_weight_bytes(g.I, g.D) + (int64_t)strip * mx4_strip_bytes(g.D);
  const bool real = 16 * strip < g.I;  // h's columns are padded to whole blocks, with zeros
  auto fetch = [&](MoeChunk (&w)[2], int c) {
    load_chunk(w[0], real ? g.wg + at + (int64_t)kChunkBytes * c : nullptr, blocks - 16 * c, lane);
    load_chunk(w[1], real ? g.wu + at + (int64_t)kChunkBytes * c : nullptr, blocks - 16 * c, lane);
  };
  MoeChunk w[2], wn[2];
  int c0 = wave;
  if (c0 < chunks) fetch(w, c0);
  const int members = __popcll(who);
  if (wave == 0) {
    place[lane] = o.place[64 * slot + lane];
    if ((who >> lane) & 1) tok[__popcll(who & ((uint64_t(1) << lane) - 1))] = lane;
  }
  __syncthreads();
  buf_t xb[XP];
  part_buffers<XP>(xb, o.x, g.T, Dp);
  for (int r0 = 0; r0 < members; r0 += 16) {
    const int row = r0 + l16;
    const int xoff = row < members ? 2 * tok[row] * Dp : kNowhere;
    f32x4_t acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    if (r0 > 0 && wave < chunks) fetch(w, wave);
    for (int c = wave; c < chunks; c += kUpWaves) {
      const int nb = blocks - 16 * c;
      MoeRows<XP> a[2];
      a[0].load(xb, xoff + 1024 * c, 0, nb, lane);
      if (c + kUpWaves < chunks) fetch(wn, c + kUpWaves);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j < 3) a[(j + 1) & 1].load(xb, xoff + 1024 * c, j + 1, nb, lane);
#pragma unroll
        for (int p = 0; p < 2; ++p) multiply<XP>(acc[p], a[j & 1], w[p].c[j], scale_f32((w[p].s >> (8 * j)) & 255));
      }
      w[0] = wn[0], w[1] = wn[1];
    }
    if (r0 > 0) __syncthreads();
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int q = 0; q < 4; ++q) sums[wave][p][4 * quad + q][l16] = acc[p][q];
    __syncthreads();
    const int rr = threadIdx.x / 16, col = threadIdx.x % 16;
    if (r0 + rr < members) {
      const int t = tok[r0 + rr];
      const uint2 pl = place[t];
      float gv = 0.f, uv = 0.f;
#pragma unroll
      for (int q = 0; q < kUpWaves; ++q) gv += sums[q][0][rr][col], uv += sums[q][1][rr][col];
      float h = 0.f;
      with_act(g.act, [&](auto a) {
        float d;
        h = act_parts<decltype(a)::value>(gv, &d) * uv * __builtin_bit_cast(float, pl.y);
      });
      uint16_t p[HP];
      parts_of<HP>(16 * strip + col < g.I ? h : 0.f, p);  // the padding is 0 whatever x is
#pragma unroll
      for (int q = 0; q < HP; ++q)
        o.h[((int64_t)q * g.T * g.top_k + t * g.top_k + (int)pl.x) * Ip + 16 * strip + col] = p[q];
    }
  }
}

// ---- second half ---------------------------------------------------------------
// A workgroup: COLS columns of y (16, or 8 or 4 of a strip where strips are too few to occupy the chip), all
// experts; the waves take shares of (expert, chunk), one after the other.  An expert's rows are added to the
// wave's sums of its tokens in LDS, the waves' sums in their order at the end.
constexpr int kDownWaves = 16;

template <int TMAX, int HP>
__global__ __launch_bounds__(64 * kDownWaves) void moe_down_kernel(MoeArgs g, MoeBufs o, int Ip, int slots, int cols) {
  __shared__ float sums[kDownWaves][TMAX][17];
  __shared__ int toks[kDownWaves][kMoeTokens];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, quad = lane >> 4;
  const int per = 16 / cols, strip = (int)blockIdx.x / per, part = (int)blockIdx.x % per;
  const bool mine = l16 / cols == part;
  const int chunks = mx4_chunks(g.I), blocks = mx4_blocks(g.I);
  int count = 0;
  for (int s = 0; s < slots; s += 64) count += __popcll(__ballot(s + lane < slots && o.slots[min(s + lane, slots - 1)] >= 0));
  for (int i = lane; i < TMAX * 17; i += 64) (&sums[wave][0][0])[i] = 0.f;
  buf_t hb[HP];
  part_buffers<HP>(hb, o.h, g.T * g.top_k, Ip);
  const int items = count * chunks;
  const int end = (int)((int64_t)items * (wave + 1) / kDownWaves);
  int it = (int)((int64_t)items * wave / kDownWaves);
  auto where = [&](int i) -> const uint8_t* {
    if (i >= end) return nullptr;
    const int s = i / chunks;
    return g.wd + (int64_t)o.slots[s] * mx4_weight_bytes(g.D, g.I) + (int64_t)strip * mx4_strip_bytes(g.I) +
           (int64_t)kChunkBytes * (i - s * chunks);
  };
  auto fetch = [&](MoeChunk& w, int i) { load_chunk(w, where(i), mine ? blocks - 16 * (i % chunks) : 0, lane); };
  MoeChunk w, wn;
  fetch(w, it);
  while (it < end) {
    const int slot = it / chunks, c0 = it - slot * chunks, c1 = min(chunks, c0 + end - it);
    const uint64_t who = o.who[slot];
    const uint2 pl = o.place[64 * slot + lane];
    const int members = __popcll(who);
    if ((who >> lane) & 1) toks[wave][__popcll(who & ((uint64_t(1) << lane) - 1))] = lane | ((int)pl.x << 8);
    for (int r0 = 0; r0 < members; r0 += 16) {
      const int row = r0 + l16;
      const int tk = row < members ? toks[wave][row] : 0;
      const int hoff = row < members ? 2 * ((tk & 255) * g.top_k + (tk >> 8)) * Ip : kNowhere;
      const bool again = r0 + 16 < members;
      f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
      for (int c = c0; c < c1; ++c) {
        const int nb = blocks - 16 * c;
        MoeRows<HP> a[2];
        a[0].load(hb, hoff + 1024 * c, 0, nb, lane);
        const int next = c + 1 < c1 ? it + c + 1 - c0 : (again ? it : it + c1 - c0);
        fetch(wn, next);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j < 3) a[(j + 1) & 1].load(hb, hoff + 1024 * c, j + 1, nb, lane);
          multiply<HP>(acc, a[j & 1], w.c[j], scale_f32((w.s >> (8 * j)) & 255));
        }
        w = wn;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = r0 + 4 * quad + q;
        if (r < members) sums[wave][toks[wave][r] & 255][l16] += acc[q];
      }
    }
    it += c1 - c0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < g.T * 16; i += 64 * kDownWaves) {
    const int t = i / 16, col = i % 16, n = 16 * strip + col;
    if (n >= g.D || col / cols != part) continue;
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < kDownWaves; ++q) v += sums[q][t][col];
    with_y(g.y, g.y_dtype, [&](auto* yt) {
      typedef typename std::remove_pointer<decltype(yt)>::type Y;
      yt[(int64_t)t * g.ldy + n] = (Y)v;
    });
  }
}

// ---------------------------------------------------------------- host side
MoePlan plan_moe(int T, int D, int I, int E, int top_k, int x_dtype, int y_dtype) {
  MoePlan p{};
  p.xparts = x_dtype == YF32 ? 3 : x_dtype == XF16 ? 2 : 1;
  p.hparts = y_dtype == YF32 ? 3 : 2;
  p.Dp = (int)round_up(D, kBlock);
  p.Ip = (int)round_up(I, kBlock);
  p.slots = (int64_t)T * top_k < E ? T * top_k : E;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (size_t)round_up((int64_t)bytes, 256);
    return o;
  };
  p.list = take((size_t)p.slots * 4);
  p.who = take((size_t)p.slots * 8);
  p.place = take((size_t)p.slots * 64 * 8);
  p.x = take((size_t)p.xparts * T * p.Dp * 2);
  p.h = take((size_t)p.hparts * T * top_k * p.Ip * 2);
  p.bytes = at;
  return p;
}

template <int XP, int HP> static hipError_t moe_t(const MoeArgs& a, const MoePlan& p, const MoeBufs& o, hipStream_t s) {
  const int units = a.T * (p.Dp / 8), most = 64;
  const int xg = (units + 64 * kRouteWaves - 1) / (64 * kRouteWaves);
  hipError_t e = launch_kernel(moe_route_kernel<XP>, dim3((unsigned)(1 + (xg < most ? xg : most))), dim3(64 * kRouteWaves), s,
                               a, o, p.Dp, p.slots);
  if (e != hipSuccess) return e;
  e = launch_kernel(moe_up_kernel<XP, HP>, dim3((unsigned)(p.Ip / 16), (unsigned)p.slots), dim3(64 * kUpWaves), s, a, o,
                    p.Dp, p.Ip);
  if (e != hipSuccess) return e;
  const int strips = (a.D + 15) / 16, cols = strips >= 192 ? 16 : strips >= 96 ? 8 : 4;
  return launch_kernel(a.T <= 16 ? moe_down_kernel<16, HP> : moe_down_kernel<64, HP>,
                       dim3((unsigned)(strips * (16 / cols))), dim3(64 * kDownWaves), s, a, o, p.Ip, p.slots, cols);
}

template <int XP> static hipError_t moe_h(const MoeArgs& a, const MoePlan& p, const MoeBufs& o, hipStream_t s) {
  return p.hparts == 3 ? moe_t<XP, 3>(a, p, o, s) : moe_t<XP, 2>(a, p, o, s);
}

hipError_t launch_mx4_moe(const MoeArgs& a, const MoePlan& p, hipStream_t s) {
  char* ws = static_cast<char*>(a.ws);
  const MoeBufs o{reinterpret_cast<int*>(ws + p.list), reinterpret_cast<uint64_t*>(ws + p.who),
                  reinterpret_cast<uint2*>(ws + p.place), reinterpret_cast<uint16_t*>(ws + p.x),
                  reinterpret_cast<uint16_t*>(ws + p.h)};
  switch (p.xparts) {
    case 1: return moe_h<1>(a, p, o, s);
    case 2: return moe_h<2>(a, p, o, s);
  }
  return moe_h<3>(a, p, o, s);
}

}  // namespace qmm
