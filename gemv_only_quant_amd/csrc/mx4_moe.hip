// mx4_moe.hip -- a mixture-of-experts layer for up to 64 tokens, experts' weights
// in packed microscaled 4-bit codes, activations as they are.
//
//   h[t][j] = w[t][j] act(Wg_e x[t]) * (Wu_e x[t]),  y[t] = sum_j Wd_e h[t][j]
//
// Bound by reading the weights of the experts that some token chose: once for each 32 tokens of an expert (bf16 x), 16 (fp16) or
// 10 to 15 (fp32, and h), which is what a workgroup's products hold.  The products run on the 16-bit matrix cores: a
// code times its scale is exact in bf16, whose exponents reach as far as the scales', and an activation of more bits is a
// sum of bf16 parts (fp16: 2, fp32 and h: 3, exact), rows of the product beside each other, whose sums are
// added in fp32.  The other rows are an expert's further tokens, so most of the time parts cost nothing.
//
// Launches: the tokens' choices, and x as parts; the first half, h; the second, rows of y of each choice; their sum.  What
// differs is how rows and weights come to a wave (us from one launch to the next, bf16 if not said):
//
//  few     up to 4 tokens: each workgroup of the first half makes the choices itself, one of the second has its columns of y
//          whole.  Two launches, bound by their latencies: one token, 8 of 128 experts of 2048 x 768, 14.0 (16.1 with the
//          next forms' second half)
//  held    many columns for each CU: a workgroup holds an expert's rows in LDS, a wave has whole tiles and no barrier between
//          them.  64 tokens, 64 experts of 2048 x 1408, 6 each, fp16: 87 (3.4 TB/s of weights; second half by the
//          next form 97); 16 tokens, 8 experts of 4096 x 14336, 2 each: 142 (5.2 TB/s; 154)
//  other   K over a workgroup's waves, rows through each wave's own LDS: 5 tokens, 16 experts of 1001 x 777, 4 each, fp32: 18
#include <math.h>

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

// Of h, whatever y's type: the fp32 values as they are.  (2 parts are 16 bits: where nearly equal values of h meet with
// opposite signs, what is left would be off by up to 2^-16 of them, which a 16-bit y shows.)
constexpr int kHParts = 3;
template <int XP> constexpr int kTypeOfParts = XP == 1 ? XBF16 : XP == 2 ? XF16 : YF32;  // of x

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

// Activations lie in rows of whole chunks, a chunk's 512 values in the order in which the matrix cores
// take them: eight values i of blocks 4 q + j at 128 j + 32 i + 8 q.
__device__ __forceinline__ int operand_order(int k) {
  const int b = k / 32;
  return (k & ~511) + 128 * (b & 3) + 32 * ((k >> 3) & 3) + 8 * ((b >> 2) & 3) + (k & 7);
}

// What the first launch leaves for the others, in the workspace.
struct MoeBufs {
  int* ids;        // (T, top_k) experts, -1: none
  float* w;        // and their weights
  uint32_t* done;  // workgroups that have left their part of a strip of y, 0 at first
  uint16_t* x;     // (parts, T, Dp): x as a sum of bf16 parts
  uint16_t* h;     // (parts, T top_k, Ip)
  float* z;        // (T top_k, Dz): a token's rows of each of its experts
};

// A wave's choice among up to 64 HELD experts, by the top_k largest logits of token t, the lowest index first of equal
// ones: ids and w, t top_k on, in the order of indices.
template <int HELD> __device__ __forceinline__ void choose_of(const MoeArgs& g, int t, int lane, int* ids, float* w) {
  const int k = g.top_k, size = g.logits_dtype == YF32 ? 4 : 2;
  // orders of expert 64 i + lane's logits; 0: there is none, or -infinity.  (All loads before the first use.)
  uint32_t held[HELD];
  const buf_t row = make_buf(static_cast<const char*>(g.logits) + (int64_t)t * g.ldl * size, (uint32_t)(g.E * size));
  if (size == 4) {
#pragma unroll
    for (int i = 0; i < HELD; ++i) held[i] = __builtin_amdgcn_raw_buffer_load_b32(row, 4 * (64 * i + lane), 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < HELD; ++i) held[i] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(row, 2 * (64 * i + lane), 0, 0);
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    const float v = g.logits_dtype == YF32   ? __builtin_bit_cast(float, held[i])
                    : g.logits_dtype == XF16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)held[i])
                                             : __builtin_bit_cast(float, held[i] << 16);
    held[i] = 64 * i + lane >= g.E || v == -__builtin_inff() ? 0 : order_of(v);
    top = held[i] > top ? held[i] : top;
  }
  top = wave_max_u32(top);
  auto at_least = [&](uint32_t v) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < HELD; ++i) n += __popcll(__ballot(held[i] >= v));
    return n;
  };
  // The largest number that k orders reach, bit by bit from the highest, or one that k reach and no more: some 14 steps, where
  // k searches for the largest that is left took 8 of 128 experts 3.7 us.
  uint32_t least = 0;
  bool more = at_least(1) > k;  // than k reach it
  if (!more) least = 1;
  for (uint32_t bit = 1u << 31; more && bit != 0; bit >>= 1) {
    const int n = at_least(least | bit);
    if (n >= k) least |= bit, more = n > k;
  }
  // those above it, and of those at it as many as are left, the lowest indices first
  const int equal = more ? k - (least == ~0u ? 0 : at_least(least + 1)) : k;
  // (NaN, and infinity less infinity: the whole row)
  const float first = value_of(top);
  const bool finite = first - first == 0.f;
  auto share = [&](uint32_t v) { return finite ? exp_f32(value_of(v) - first) : __builtin_nanf(""); };
  const uint64_t before = (uint64_t(1) << lane) - 1;
  float p[HELD], sum = 0.f;
  int at[HELD], taken = 0, met = 0;
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    const uint64_t ties = __ballot(held[i] == least);
    const bool take = held[i] > least || (held[i] == least && met + __popcll(ties & before) < equal);
    const uint64_t takes = __ballot(take);
    at[i] = take ? taken + __popcll(takes & before) : -1;
    met += __popcll(ties), taken += __popcll(takes);
    p[i] = take || (!g.renormalize && held[i] != 0) ? share(held[i]) : 0.f;
    sum += p[i];
  }
  sum = wave_sum(sum);
#pragma unroll
  for (int i = 0; i < HELD; ++i)
    if (at[i] >= 0) ids[t * k + at[i]] = 64 * i + lane, w[t * k + at[i]] = p[i] / sum;
  if (lane >= taken && lane < k) ids[t * k + lane] = -1, w[t * k + lane] = 0.f;
}

// A wave's choice for token t: its experts and weights to ids and w, t top_k on.
__device__ __forceinline__ void choose(const MoeArgs& g, int t, int lane, int* ids, float* w) {
  const int k = g.top_k;
  if (g.logits != nullptr) {
    if (g.E <= 128) choose_of<2>(g, t, lane, ids, w);
    else if (g.E <= 256) choose_of<4>(g, t, lane, ids, w);
    else choose_of<kMoeExperts / 64>(g, t, lane, ids, w);
  } else if (lane < k) {
    const int64_t i = (int64_t)t * k + lane;
    const int64_t e = g.ids_size == 8 ? static_cast<const int64_t*>(g.ids)[i] : static_cast<const int32_t*>(g.ids)[i];
    ids[i] = e >= 0 && e < g.E ? (int)e : -1;
    w[i] = as_f32(g.weights, i, g.weights_dtype);
  }
}

// A wave for each token's choice (the first T), then threads for x as parts.
template <int XP>
__global__ __launch_bounds__(256) void moe_route_kernel(MoeArgs g, MoeBufs o, int strips, int Dp) {
  const int tid = (int)blockIdx.x * 256 + (int)threadIdx.x, lane = threadIdx.x & 63;
  const int t = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int i = tid; i < strips; i += (int)gridDim.x * 256) o.done[i] = 0;
  const int groups = (g.T + 3) / 4;  // workgroups that choose
  if ((int)blockIdx.x < groups) {
    if (t < g.T) choose(g, t, lane, o.ids, o.w);
    return;
  }
  constexpr int XT = kTypeOfParts<XP>;
  const int units = Dp / 8;
  for (int u = tid - 256 * groups; u < g.T * units; u += ((int)gridDim.x - groups) * 256) {
    const int r = u / units, i = 8 * (u - r * units);
    float f[8];
    Raw8<XT> raw = take8<XT, false>(static_cast<const typename Elem<XT>::type*>(g.x) + (int64_t)r * g.ldx, i, g.D);
    settle8<XT, false>(raw, i, g.D);
    floats8<XT>(raw, f);
    uint16_t p[8][XP];
#pragma unroll
    for (int j = 0; j < 8; ++j) parts_of<XP>(f[j], p[j]);
#pragma unroll
    for (int q = 0; q < XP; ++q) {
      u32x4_t v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = p[2 * j][q] | ((uint32_t)p[2 * j + 1][q] << 16);
      *reinterpret_cast<u32x4_t*>(o.x + ((int64_t)q * g.T + r) * Dp + operand_order(i)) = v;
    }
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

// Buffers of the parts of `rows` rows of `ld` bf16 values.
template <int P> __device__ __forceinline__ void part_buffers(buf_t (&b)[P], const uint16_t* p, int rows, int ld) {
#pragma unroll
  for (int q = 0; q < P; ++q) b[q] = make_buf(p + (int64_t)q * rows * ld, 2u * (uint32_t)rows * (uint32_t)ld);
}

// An expert's tokens, from the slot of a workgroup: expert `slot` itself, or (`pairs`) the expert of
// place `slot` of all tokens' choices unless an earlier place has it too.
struct MoeGroup {
  int e;          // -1: none
  uint64_t who;   // its tokens, a bit each
  int place;      // lane t: the first of token t's places that holds it, or -1
  float w;        // and the sum of all such places' weights
};
__device__ __forceinline__ MoeGroup group_of(const MoeBufs& o, int slot, bool pairs, int T, int k, int lane) {
  // (what does not depend on the expert is requested first, so that the loads' latencies overlap)
  constexpr int HELD = 8;
  const int* ids = o.ids + (lane < T ? lane * k : 0);
  const float* w = o.w + (lane < T ? lane * k : 0);
  int own[HELD];
  float ow[HELD];
#pragma unroll
  for (int j = 0; j < HELD; ++j) own[j] = ids[j < k ? j : 0], ow[j] = w[j < k ? j : 0];
  MoeGroup m;
  m.e = slot;
  if (pairs) {
    int earlier = lane < slot ? o.ids[lane] : -1;
    m.e = __builtin_amdgcn_readfirstlane(o.ids[slot]);
    bool before = m.e < 0 || earlier == m.e;
    for (int p = 64 + lane; p < slot; p += 64) before |= o.ids[p] == m.e;
    if (__ballot(before) != 0) m.e = -1;
  }
  m.place = -1;
  m.w = 0.f;
  if (lane < T && m.e >= 0) {
#pragma unroll
    for (int j = 0; j < HELD; ++j) {
      const bool same = j < k && own[j] == m.e;
      m.place = same && m.place < 0 ? j : m.place;
      m.w += same ? ow[j] : 0.f;
    }
    for (int j = HELD; j < k; ++j) {
      const bool same = ids[j] == m.e;
      m.place = same && m.place < 0 ? j : m.place;
      m.w += same ? w[j] : 0.f;
    }
  }
  m.who = __ballot(m.place >= 0);
  if (m.who == 0) m.e = -1;
  return m;
}

// A workgroup's products: tiles (pairs of 16 columns of an expert) one after the other, in each of which a wave
// takes chunks of K in turn; put(tile, sums) is called by all waves when a tile's sums of a wave are
// complete: acc[g][p] of rows RG g .. of `members` and of column half p.
// The rows of a chunk come as whole lines, 1 KiB a load, and through the wave's own part of LDS to the
// operands' places (straight from memory a load touches 16 lines for 256 bytes: 16 tokens, 8 experts of
// 4096 x 14336, second half 103 us).  LDS holds RG rows in all their parts; the next ones are on
// their way while these are multiplied, and behind them the next chunk's weights (the next tile's
// after a tile's last): loads return in order, and what is waited for first goes first.
constexpr int kRowBytes = 1024 + 16;  // of LDS: neighbouring rows start in different banks
constexpr int kMoeWaves = 4;
template <int P> constexpr int kRowGroup = 16 / P;  // rows of which a wave holds all P parts

struct MoeLds {
  char rows[kMoeWaves][16 * kRowBytes];
  float sums[kMoeWaves][2][16][17];
};

// Where rows come from.  Parts: rows of bf16 parts in operand order; lane r has the offset of row r.
template <int P> struct Parts {
  static constexpr int RG = kRowGroup<P>;
  buf_t parts[P];
  int offs, members, blocks, lane;
  char* lds;
  u32x4_t v[P][RG];
  // row group g of chunk c to registers: 16 bytes of lane L are 8 values of block 4 (L % 4) + L / 16
  __device__ __forceinline__ void request(int g, int c) {
    const int at = 4 * (lane & 3) + (lane >> 4) < blocks - 16 * c ? 16 * lane + 1024 * c : kNowhere;
#pragma unroll
    for (int r = 0; r < RG; ++r) {
      if (r % 4 == 0 && RG * g + r >= members) break;
      const int row = __builtin_amdgcn_readlane(offs, RG * g + r);
#pragma unroll
      for (int q = 0; q < P; ++q) v[q][r] = __builtin_amdgcn_raw_buffer_load_b128(parts[q], at, row, 0);
    }
  }
  // and from there to LDS
  __device__ __forceinline__ void leave(int g) {
#pragma unroll
    for (int r = 0; r < RG; ++r) {
      if (r % 4 == 0 && RG * g + r >= members) break;
#pragma unroll
      for (int q = 0; q < P; ++q) *reinterpret_cast<u32x4_t*>(lds + (RG * q + r) * kRowBytes + 16 * lane) = v[q][r];
    }
  }
};
// x itself, up to 4 tokens: 8 values a lane, made parts on the way to LDS.  VEC: rows of whole 16 bytes.
template <int XT, int P, bool VEC> struct Values {
  static constexpr int RG = kRowGroup<P>, SIZE = XT == YF32 ? 4 : 2;
  static_assert(RG >= 4, "rows");
  typedef typename Elem<XT>::type T;
  const T* x;
  int64_t ldx;
  buf_t rows[4];
  int members, lane, K, k;  // k: this lane's first value of those requested
  char* lds;
  Raw8<XT> v[4];
  __device__ __forceinline__ Values(const MoeArgs& g, int lane, char* lds)
      : x(static_cast<const T*>(g.x)), ldx(g.ldx), members(g.T), lane(lane), K(g.D), lds(lds) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      rows[r] = make_buf(x + (r < g.T ? r : 0) * ldx, r < g.T ? (uint32_t)(K * SIZE) : 0u);
  }
  __device__ __forceinline__ void request(int, int c) {
    k = 512 * c + 8 * lane;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (r >= members) break;
      if constexpr (VEC) v[r] = load8<XT, true>(rows[r], k);
      else v[r] = take8<XT, false>(x + r * ldx, k, K);
    }
  }
  __device__ __forceinline__ void leave(int) {
    // 8 values i = lane % 4 of block lane / 4 = 4 q + j
    char* to = lds + 256 * ((lane >> 2) & 3) + 64 * (lane & 3) + 16 * (lane >> 4);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (r >= members) break;
      settle8<XT, VEC>(v[r], k, K);
      if constexpr (P == 1) {
        *reinterpret_cast<u32x4_t*>(to + r * kRowBytes) = v[r].w[0];
      } else {
        float f[8];
        floats8<XT>(v[r], f);
        uint16_t p[8][P];
#pragma unroll
        for (int j = 0; j < 8; ++j) parts_of<P>(f[j], p[j]);
#pragma unroll
        for (int q = 0; q < P; ++q) {
          u32x4_t o;
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = p[2 * j][q] | ((uint32_t)p[2 * j + 1][q] << 16);
          *reinterpret_cast<u32x4_t*>(to + (RG * q + r) * kRowBytes) = o;
        }
      }
    }
  }
};

template <int P, int G, class Source, class Fetch, class Put>
__device__ __forceinline__ void sweep(Source& rows, int members, int wave, int tile, int tiles, int chunks, char* lds, int lane,
                                      Fetch&& fetch, Put&& put) {
  constexpr int RG = kRowGroup<P>;
  const int l16 = lane & 15, quad = lane >> 4;
  MoeChunk w[2], wn[2];
  fetch(w, tile, wave);
  // rows that fit LDS at once and serve every tile stay there
  const bool stay = members <= RG && chunks <= kMoeWaves;
  bool staged = false;
  for (; tile < tiles; ++tile) {
    f32x4_t acc[G][2];
#pragma unroll
    for (int g = 0; g < G; ++g) acc[g][0] = acc[g][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int c = wave; c < chunks; c += kMoeWaves) {
      const bool more = c + kMoeWaves < chunks;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (RG * g >= members) break;
        const bool last = g + 1 == G || RG * (g + 1) >= members;
        if (!staged) {
          rows.leave(g);
          staged = stay;
          if (!last) rows.request(g + 1, c);
          else if (!stay && (more || tile + 1 < tiles)) rows.request(0, more ? c + kMoeWaves : wave);
        }
        if (last) fetch(wn, more ? tile : tile + 1, more ? c + kMoeWaves : wave);
        // a row's parts are rows of the product, RG apart, and their sums are added afterwards
        const char* from = lds + min(l16, P * RG - 1) * kRowBytes + 16 * quad;
        // (weights are converted anew for every group: kept, the operands would fill the registers)
#pragma unroll
        for (int j = 0; j < 4; ++j) asm volatile("" : "+v"(w[0].c[j]), "+v"(w[1].c[j]));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float s0 = scale_f32((w[0].s >> (8 * j)) & 255), s1 = scale_f32((w[1].s >> (8 * j)) & 255);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bf16x8_t b0 = __builtin_bit_cast(bf16x8_t, bf16_of_codes(w[0].c[j][i], s0));
            const bf16x8_t b1 = __builtin_bit_cast(bf16x8_t, bf16_of_codes(w[1].c[j][i], s1));
            const bf16x8_t a = __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4_t*>(from + 256 * j + 64 * i));
            acc[g][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b0, acc[g][0], 0, 0, 0);
            acc[g][1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b1, acc[g][1], 0, 0, 0);
          }
        }
      }
      w[0] = wn[0], w[1] = wn[1];
    }
    put(tile, acc);
  }
}

// The waves' sums of row group i to LDS, where all may read them afterwards.  The first barrier keeps the
// readers of what was there apart.
template <int G>
__device__ __forceinline__ void meet(MoeLds& lds, const f32x4_t (&acc)[G][2], int i, int wave, int lane) {
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int q = 0; q < 4; ++q) lds.sums[wave][p][4 * (lane >> 4) + q][lane & 15] = acc[i][p][q];
  __syncthreads();
}

// Column `col` of half `p` of row rr of the group that met: its parts' sums of all waves, the smallest part first.
template <int P> __device__ __forceinline__ float met(const MoeLds& lds, int p, int rr, int col) {
  float v = 0.f;
#pragma unroll
  for (int i = P; i-- > 0;)
#pragma unroll
    for (int q = 0; q < kMoeWaves; ++q) v += lds.sums[q][p][kRowGroup<P> * i + rr][col];
  return v;
}

// Where an expert's rows fit LDS whole and there are tiles enough, a wave has whole tiles instead: nothing is left to
// add across waves, and no barrier stands between a wave and its next weights.
constexpr int kHeldWaves = 12, kHeldBytes = 30 * (5 * 1024 + 16);
constexpr int64_t kRangesBytes = 1 << 28;  // of z, if more than one range of chunks is held
// A product's rows, of each its P parts, and how many such groups there may be.
template <int P> constexpr int kHeldRows = P == 1 ? 16 : P == 2 ? 8 : 5;
template <int P> constexpr int kHeldGroups = P == 3 ? 3 : 2;
template <int P> constexpr int held_chunks(int groups) { return (kHeldBytes / (P * kHeldRows<P> * groups) - 16) / 1024; }  // of a row
// Part q of row r of a group is this row of the product.  Lanes of a quad have rows 4 quad .. + 3 of the sums: 3 parts of rows
// 0 to 3 lie in as many quads, those of row 4 in the last quad beside each other.
template <int P> __device__ __forceinline__ int held_slot(int r, int q) {
  return P == 3 ? (r == 4 ? 12 + q : 4 * q + r) : kHeldRows<P> * q + r;
}
// The row whose whole sum a lane has at place i of its four; kHeldRows or more: none.
template <int P> __device__ __forceinline__ int held_row(int quad, int i) {
  return P == 3 ? (quad == 0 ? i : quad == 3 && i == 0 ? 4 : kHeldRows<P>) : 4 * quad + i;
}

struct HeldLds {
  char rows[kHeldBytes];
  int row[kMoeTokens];    // of members: token top_k + place
  int tok[kMoeTokens];
  float wt[kMoeTokens];
};

// Chunks c0 .. of `rows` rows of bf16 parts in operand order to LDS, a chunk a turn; first() is called when the first ones
// are requested.
template <int P, class Offset, class First>
__device__ __forceinline__ void hold_rows(HeldLds& lds, const buf_t (&parts)[P], int rows, int ld, int c0, int chunks,
                                          int blocks, int wave, int lane, Offset&& offset, First&& first) {
  constexpr int RG = kHeldRows<P>, AHEAD = 4;
  const int turns = rows * P * chunks;
  // t / chunks, exact for what fits LDS (fewer than 2^16 / chunks turns)
  const uint32_t inverse = 65535u / (uint32_t)chunks + 1;
  auto row_of = [&](int t) { return (int)((uint32_t)t * inverse >> 16); };
  u32x4_t v[AHEAD];
  auto get = [&](int t) {
    const int r = row_of(t), m = r / P, q = r % P, c = t - r * chunks;
    const bool ok = t < turns && 4 * (lane & 3) + (lane >> 4) < blocks - 16 * (c0 + c);
    const int at = ok ? 1024 * (c0 + c) + 16 * lane : kNowhere, row = t < turns ? offset(m) : 0;
    u32x4_t x = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (i == q) x = __builtin_amdgcn_raw_buffer_load_b128(parts[i], at, row, 0);
    return x;
  };
  auto put = [&](int t, const u32x4_t& x) {
    const int r = row_of(t), m = r / P, q = r % P, c = t - r * chunks;
    const int to = (P * RG * (m / RG) + held_slot<P>(m % RG, q)) * ld + 1024 * c + 16 * lane;
    if (t < turns) *reinterpret_cast<u32x4_t*>(lds.rows + to) = x;
  };
  for (int t = wave; t == wave || t < turns; t += AHEAD * kHeldWaves) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) v[i] = get(t + i * kHeldWaves);
    if (t == wave) first();
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) put(t + i * kHeldWaves, v[i]);
  }
  __syncthreads();
}

// The tiles tile, tile + kHeldWaves .. of a wave, their weights in two sets of registers in turn; put(tile, sums of rows).
template <int P, int G> struct HeldSweep {
  MoeChunk w[2][2];
  int t, c, tn, cn;  // the unit whose weights come first, and the one requested last
  template <class Fetch> __device__ __forceinline__ void begin(int tile, int tiles, int chunks, Fetch&& fetch) {
    t = tn = tile, c = cn = 0;
    fetch(w[0], tn, cn);
    after(tn, cn, chunks);
    fetch(w[1], tn, cn);
  }
  static __device__ __forceinline__ void after(int& t, int& c, int chunks) {
    if (++c == chunks) c = 0, t += kHeldWaves;
  }
  template <class Fetch, class Put>
  __device__ __forceinline__ void run(const char* rows, int ld, int groups, int tiles, int chunks, int lane, Fetch&& fetch,
                                      Put&& put) {
    f32x4_t acc[G][2] = {};
    constexpr int ROWS = P * kHeldRows<P>;
    const char* from0 = rows + min(lane & 15, ROWS - 1) * ld + 16 * (lane >> 4);
    auto use = [&](const MoeChunk (&m)[2]) {
      const char* from = from0 + 1024 * c;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float s0 = scale_f32((m[0].s >> (8 * j)) & 255), s1 = scale_f32((m[1].s >> (8 * j)) & 255);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bf16x8_t b0 = __builtin_bit_cast(bf16x8_t, bf16_of_codes(m[0].c[j][i], s0));
          const bf16x8_t b1 = __builtin_bit_cast(bf16x8_t, bf16_of_codes(m[1].c[j][i], s1));
#pragma unroll
          for (int g = 0; g < G; ++g) {
            if (g > 0 && g >= groups) break;
            const char* at = from + ROWS * g * ld + 256 * j + 64 * i;
            const bf16x8_t a = __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const u32x4_t*>(at));
            acc[g][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b0, acc[g][0], 0, 0, 0);
            acc[g][1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b1, acc[g][1], 0, 0, 0);
          }
        }
      }
      if (c == chunks - 1) {
        // a row's parts lie in different lanes of a column
#pragma unroll
        for (int g = 0; g < G; ++g) {
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const float last = acc[g][p][0] + (acc[g][p][1] + acc[g][p][2]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float v = acc[g][p][r];
              if (P == 2) acc[g][p][r] = v + __shfl_xor(v, 32, 64);
              if (P == 3) acc[g][p][r] = v + (__shfl(v, (lane & 15) + 16, 64) + __shfl(v, (lane & 15) + 32, 64));
            }
            if (P == 3 && lane >= 48) acc[g][p][0] = last;
          }
        }
        put(t, acc);
#pragma unroll
        for (int g = 0; g < G; ++g) acc[g][0] = acc[g][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
      after(t, c, chunks);
    };
    while (t < tiles) {
      use(w[0]);
      after(tn, cn, chunks);
      fetch(w[0], tn, cn);
      if (t >= tiles) break;
      use(w[1]);
      after(tn, cn, chunks);
      fetch(w[1], tn, cn);
    }
  }
};

// ---- first half ----------------------------------------------------------------
// Column threadIdx.x % 16 of strip t of h, from the waves' sums of row rr, for `place` of token `tok`.
template <int XP>
__device__ __forceinline__ void put_hidden(const MoeArgs& g, const MoeBufs& o, const MoeLds& lds, int rr, int t, int tok,
                                           int place, float wt, int Ip) {
  const int col = threadIdx.x % 16;
  const float gv = met<XP>(lds, 0, rr, col), uv = met<XP>(lds, 1, rr, col);
  float h = 0.f;
  with_act(g.act, [&](auto a) {
    float d;
    h = act_parts<decltype(a)::value>(gv, &d) * uv * wt;
  });
  uint16_t p[kHParts];
  parts_of<kHParts>(16 * t + col < g.I ? h : 0.f, p);  // the padding is 0 whatever x is
  const int row = tok * g.top_k + place, at = operand_order(16 * t + col);
#pragma unroll
  for (int q = 0; q < kHParts; ++q) o.h[((int64_t)q * g.T * g.top_k + row) * Ip + at] = p[q];
}

// A workgroup: `per` strips of 16 columns of h of one expert.
template <int XP, int G>
__global__ __launch_bounds__(64 * kMoeWaves, 2) void moe_up_kernel(MoeArgs g, MoeBufs o, int Dp, int Ip, int pairs, int per) {
  __shared__ MoeLds lds;
  __shared__ int tok[kMoeTokens], place[kMoeTokens];
  __shared__ float wt[kMoeTokens];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const MoeGroup m = group_of(o, (int)blockIdx.y, pairs != 0, g.T, g.top_k, lane);
  if (m.e < 0) return;
  const int chunks = mx4_chunks(g.D), blocks = mx4_blocks(g.D);
  const int strips = 2 * mx4_blocks(g.I);  // h's columns are padded to whole blocks, with zeros
  const int tile = per * (int)blockIdx.x, tiles = min(tile + per, strips);
  const int64_t strip_bytes = mx4_strip_bytes(g.D), at = (int64_t)m.e * mx4_weight_bytes(g.I, g.D);
  auto fetch = [&](MoeChunk (&w)[2], int t, int c) {
    const bool ok = t < tiles && 16 * t < g.I && c < chunks;
    const int64_t to = at + t * strip_bytes + (int64_t)kChunkBytes * c;
    load_chunk(w[0], ok ? g.wg + to : nullptr, blocks - 16 * c, lane);
    load_chunk(w[1], ok ? g.wu + to : nullptr, blocks - 16 * c, lane);
  };
  const int members = __popcll(m.who);
  if (wave == 0 && m.place >= 0) {
    const int r = __popcll(m.who & ((uint64_t(1) << lane) - 1));
    tok[r] = lane, place[r] = m.place, wt[r] = m.w;
  }
  __syncthreads();
  constexpr int RG = kRowGroup<XP>;
  for (int r0 = 0; r0 < members; r0 += G * RG) {
    Parts<XP> rows;
    part_buffers<XP>(rows.parts, o.x, g.T, Dp);
    rows.offs = r0 + lane < members ? 2 * tok[r0 + lane] * Dp : 0;
    rows.members = members - r0, rows.blocks = blocks, rows.lane = lane, rows.lds = lds.rows[wave];
    if (wave < chunks) rows.request(0, wave);
    auto put = [&](int t, const f32x4_t (&acc)[G][2]) {
#pragma unroll
      for (int i = 0; i < G; ++i) {
        if (r0 + RG * i >= members) break;
        meet<G>(lds, acc, i, wave, lane);
        const int rr = threadIdx.x / 16, r = r0 + RG * i + rr;
        if (rr < RG && r < members) put_hidden<XP>(g, o, lds, rr, t, tok[r], place[r], wt[r], Ip);
      }
    };
    sweep<XP, G>(rows, members - r0, wave, tile, tiles, chunks, lds.rows[wave], lane, fetch, put);
  }
}

template <int XP, int G>
__global__ __launch_bounds__(64 * kHeldWaves) void moe_up_held_kernel(MoeArgs g, MoeBufs o, int Dp, int Ip, int pairs,
                                                                      int per) {
  __shared__ HeldLds lds;
  constexpr int RG = kHeldRows<XP>;
  const int lane = threadIdx.x & 63, quad = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const MoeGroup m = group_of(o, (int)blockIdx.y, pairs != 0, g.T, g.top_k, lane);
  if (m.e < 0) return;
  const int chunks = mx4_chunks(g.D), blocks = mx4_blocks(g.D), members = __popcll(m.who), ld = 2 * Dp + 16;
  const int strips = 2 * mx4_blocks(g.I);  // h's columns are padded to whole blocks, with zeros
  const int tile = per * (int)blockIdx.x, tiles = min(tile + per, strips);
  const int64_t strip_bytes = mx4_strip_bytes(g.D), at = (int64_t)m.e * mx4_weight_bytes(g.I, g.D);
  auto fetch = [&](MoeChunk (&w)[2], int t, int c) {
    const bool ok = t < tiles && 16 * t < g.I;
    const int64_t to = at + t * strip_bytes + (int64_t)kChunkBytes * c;
    load_chunk(w[0], ok ? g.wg + to : nullptr, blocks - 16 * c, lane);
    load_chunk(w[1], ok ? g.wu + to : nullptr, blocks - 16 * c, lane);
  };
  if (wave == 0 && m.place >= 0) {
    const int r = __popcll(m.who & ((uint64_t(1) << lane) - 1));
    lds.tok[r] = lane, lds.row[r] = lane * g.top_k + m.place, lds.wt[r] = m.w;
  }
  __syncthreads();
  buf_t parts[XP];
  part_buffers<XP>(parts, o.x, g.T, Dp);
  HeldSweep<XP, G> sweep;
  for (int r0 = 0; r0 < members; r0 += G * RG) {
    if (r0 > 0) __syncthreads();
    const int rows = min(members - r0, G * RG), groups = (rows + RG - 1) / RG;
    hold_rows<XP>(lds, parts, rows, ld, 0, chunks, blocks, wave, lane,
                  [&](int r) { return 2 * Dp * __builtin_amdgcn_readfirstlane(lds.tok[r0 + r]); },
                  [&] { sweep.begin(tile + wave, tiles, chunks, fetch); });
    sweep.run(lds.rows, ld, groups, tiles, chunks, lane, fetch, [&](int t, const f32x4_t (&acc)[G][2]) {
      const int n = 16 * t + l16;
#pragma unroll
      for (int i = 0; i < G; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int rr = held_row<XP>(quad, q), r = RG * i + rr;
          if (rr >= RG || r >= rows) continue;
          float h = 0.f;
          with_act(g.act, [&](auto a) {
            float d;
            h = act_parts<decltype(a)::value>(acc[i][0][q], &d) * acc[i][1][q] * lds.wt[r0 + r];
          });
          uint16_t p[kHParts];
          parts_of<kHParts>(n < g.I ? h : 0.f, p);  // the padding is 0 whatever x is
#pragma unroll
          for (int b = 0; b < kHParts; ++b) o.h[((int64_t)b * g.T * g.top_k + lds.row[r0 + r]) * Ip + operand_order(n)] = p[b];
        }
    });
  }
}

// The same for up to 4 tokens, with their choices made by every workgroup itself (a launch less: one token, 8 of 128 experts
// of 2048 x 768, 7.3 us for 4 and 7 by two), rows of the product
// the tokens in their order.  The first workgroup leaves the choices for the second half.
template <int XT, int XP, bool VEC>
__global__ __launch_bounds__(64 * kMoeWaves, 2) void moe_up_few_kernel(MoeArgs g, MoeBufs o, int Ip, int pairs, int per,
                                                                       int strips_y) {
  __shared__ MoeLds lds;
  __shared__ int ids[4 * kMoeTopK];
  __shared__ float ws[4 * kMoeTopK];
  const int lane = threadIdx.x & 63, k = g.top_k, slot = (int)blockIdx.y;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int chunks = mx4_chunks(g.D), blocks = mx4_blocks(g.D);
  Values<XT, XP, VEC> rows(g, lane, lds.rows[wave]);
  if (wave < chunks) rows.request(0, wave);
  if (wave < g.T) choose(g, wave, lane, ids, ws);
  __syncthreads();
  const int places = g.T * k;
  if (blockIdx.x == 0 && slot == 0) {
    for (int i = threadIdx.x; i < places; i += 64 * kMoeWaves) o.ids[i] = ids[i], o.w[i] = ws[i];
    for (int i = threadIdx.x; i < strips_y; i += 64 * kMoeWaves) o.done[i] = 0;
  }
  // the places with this workgroup's expert, a bit each
  const int e = pairs ? __builtin_amdgcn_readfirstlane(ids[slot]) : slot;
  const uint64_t same[2] = {__ballot(lane < places && ids[lane] == e), __ballot(64 + lane < places && ids[64 + lane] == e)};
  if (e < 0 || (same[0] | same[1]) == 0) return;
  const uint64_t below = slot < 64 ? same[0] & ((uint64_t(1) << slot) - 1)
                                   : same[0] | (same[1] & ((uint64_t(1) << (slot - 64)) - 1));
  if (pairs && below != 0) return;
  const int strips = 2 * mx4_blocks(g.I), tile = per * (int)blockIdx.x, tiles = min(tile + per, strips);
  const int64_t strip_bytes = mx4_strip_bytes(g.D), at = (int64_t)e * mx4_weight_bytes(g.I, g.D);
  auto fetch = [&](MoeChunk (&w)[2], int t, int c) {
    const bool ok = t < tiles && 16 * t < g.I && c < chunks;
    const int64_t to = at + t * strip_bytes + (int64_t)kChunkBytes * c;
    load_chunk(w[0], ok ? g.wg + to : nullptr, blocks - 16 * c, lane);
    load_chunk(w[1], ok ? g.wu + to : nullptr, blocks - 16 * c, lane);
  };
  sweep<XP, 1>(rows, g.T, wave, tile, tiles, chunks, lds.rows[wave], lane, fetch, [&](int t, const f32x4_t (&acc)[1][2]) {
    meet<1>(lds, acc, 0, wave, lane);
    const int r = threadIdx.x / 16, p = r * k;
    if (r >= g.T) return;
    uint64_t own = p >= 64 ? same[1] >> (p - 64) : p == 0 ? same[0] : same[0] >> p | same[1] << (64 - p);
    own &= (uint64_t(1) << k) - 1;
    if (own == 0) return;
    const int place = (int)__builtin_ctzll(own);
    float wt = 0.f;
    for (; own != 0; own &= own - 1) wt += ws[p + (int)__builtin_ctzll(own)];
    put_hidden<XP>(g, o, lds, r, t, r, place, wt, Ip);
  });
}

// ---- second half ---------------------------------------------------------------
// Whether place p of all tokens' choices has rows: that of an expert which no earlier place of its token has.
__device__ __forceinline__ bool first_place(const int* ids, int p, int k) {
  const int e = ids[p];
  bool first = e >= 0;
  for (int b = p - p % k; b < p; ++b) first = first && ids[b] != e;
  return first;
}

// Column n of a token's rows, those of places p0 .. + k - 1 that exist (valid), of each range of `stride` rows; added in
// this order.
template <bool COHERENT, class Valid>
__device__ __forceinline__ float token_sum(buf_t z, int p0, int k, int Dz, int n, int ranges, int stride, Valid&& valid) {
  float v = 0.f;
  for (int j0 = 0; j0 < k * ranges; j0 += 8) {  // 8 loads at once
    float r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int range = (j0 + j) / k, p = j0 + j - range * k;
      const int at = range < ranges && valid(p) ? 4 * ((range * stride + p0 + p) * Dz + n) : kNowhere;
      r[j] = __builtin_bit_cast(float, (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(z, at, 0, COHERENT ? kCoherent : 0));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v += r[j];
  }
  return v;
}

// A workgroup: `per` times 32 columns of one expert's rows of y.  A token's rows are added in the order of its places: for
// a few tokens (JOIN) by the last of those columns' workgroups to come, else by another launch (64 tokens, 64 experts of
// 2048 x 1408: few workgroups would be left with 23 us of additions, the launch takes 5).
template <int G, bool JOIN>
__global__ __launch_bounds__(64 * kMoeWaves, 2) void moe_down_kernel(MoeArgs g, MoeBufs o, int Ip, int pairs, int Dz, int per) {
  __shared__ MoeLds lds;
  __shared__ int tok[kMoeTokens], place[kMoeTokens];
  __shared__ uint32_t arrived;
  __shared__ bool valid[kMoeTokens * kMoeTopK];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int k = g.top_k;
  const int tile = per * (int)blockIdx.x, tiles = min(tile + per, Dz / 32);
  const MoeGroup m = group_of(o, (int)blockIdx.y, pairs != 0, g.T, k, lane);
  const buf_t zb = make_buf(o.z, 4u * (uint32_t)(g.T * k) * (uint32_t)Dz);
  if (m.e >= 0) {
    const int chunks = mx4_chunks(g.I), blocks = mx4_blocks(g.I);
    const int64_t strip_bytes = mx4_strip_bytes(g.I), at = (int64_t)m.e * mx4_weight_bytes(g.D, g.I);
    auto fetch = [&](MoeChunk (&w)[2], int t, int c) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        load_chunk(w[i], t < tiles && 32 * t + 16 * i < g.D && c < chunks
                             ? g.wd + at + (2 * t + i) * strip_bytes + (int64_t)kChunkBytes * c : nullptr,
                   blocks - 16 * c, lane);
    };
    const int members = __popcll(m.who);
    if (wave == 0 && m.place >= 0) {
      const int r = __popcll(m.who & ((uint64_t(1) << lane) - 1));
      tok[r] = lane, place[r] = m.place;
    }
    __syncthreads();
    constexpr int RG = kRowGroup<kHParts>;
    static_assert(RG <= 8, "rows that the workgroup's threads take at once");
    for (int r0 = 0; r0 < members; r0 += G * RG) {
      Parts<kHParts> rows;
      part_buffers<kHParts>(rows.parts, o.h, g.T * k, Ip);
      rows.offs = r0 + lane < members ? 2 * (tok[r0 + lane] * k + place[r0 + lane]) * Ip : 0;
      rows.members = members - r0, rows.blocks = blocks, rows.lane = lane, rows.lds = lds.rows[wave];
      if (wave < chunks) rows.request(0, wave);
      auto put = [&](int t, const f32x4_t (&acc)[G][2]) {
#pragma unroll
        for (int i = 0; i < G; ++i) {
          if (r0 + RG * i >= members) break;
          meet<G>(lds, acc, i, wave, lane);
          const int rr = threadIdx.x / 32, r = r0 + RG * i + rr, col = threadIdx.x % 32;
          if (rr >= RG || r >= members) continue;
          const float v = met<kHParts>(lds, col / 16, rr, col % 16);
          // past this XCD's L2: another XCD's workgroup may read it
          __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), zb,
                                                4 * ((tok[r] * k + place[r]) * Dz + 32 * t + col), 0, JOIN ? kCoherent : 0);
        }
      };
      sweep<kHParts, G>(rows, members - r0, wave, tile, tiles, chunks, lds.rows[wave], lane, fetch, put);
    }
  }
  if (!JOIN) return;
  // every wave's rows are in memory before the workgroup counts as arrived
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
  __syncthreads();
  if (threadIdx.x == 0)
    arrived = __hip_atomic_fetch_add(&o.done[blockIdx.x], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  if (arrived + 1 != gridDim.y) return;
  for (int i = threadIdx.x; i < g.T * k; i += 64 * kMoeWaves) valid[i] = first_place(o.ids, i, k);
  __syncthreads();
  const int n0 = 32 * tile, cols = min(32 * tiles, g.D) - n0;
  for (int i = threadIdx.x; i < cols * g.T; i += 64 * kMoeWaves) {
    const int t = i / cols, n = n0 + i % cols;
    const float v = token_sum<true>(zb, t * k, k, Dz, n, 1, 0, [&](int p) { return valid[t * k + p]; });
    with_y(g.y, g.y_dtype, [&](auto* yt) {
      typedef typename std::remove_pointer<decltype(yt)>::type Y;
      yt[(int64_t)t * g.ldy + n] = (Y)v;
    });
  }
}

template <int G>
__global__ __launch_bounds__(64 * kHeldWaves) void moe_down_held_kernel(MoeArgs g, MoeBufs o, int Ip, int pairs, int Dz, int per,
                                                                        int range) {
  __shared__ HeldLds lds;
  constexpr int RG = kHeldRows<kHParts>;
  const int lane = threadIdx.x & 63, quad = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const MoeGroup m = group_of(o, (int)blockIdx.y, pairs != 0, g.T, g.top_k, lane);
  if (m.e < 0) return;
  const int c0 = range * (int)blockIdx.z, chunks = min(range, mx4_chunks(g.I) - c0), ld = 1024 * range + 16;
  const int blocks = mx4_blocks(g.I), members = __popcll(m.who);
  const int tile = per * (int)blockIdx.x, tiles = min(tile + per, Dz / 32);
  const int64_t strip_bytes = mx4_strip_bytes(g.I), at = (int64_t)m.e * mx4_weight_bytes(g.D, g.I);
  auto fetch = [&](MoeChunk (&w)[2], int t, int c) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t to = at + (2 * t + i) * strip_bytes + (int64_t)kChunkBytes * (c0 + c);
      load_chunk(w[i], t < tiles && 32 * t + 16 * i < g.D ? g.wd + to : nullptr, blocks - 16 * (c0 + c), lane);
    }
  };
  if (wave == 0 && m.place >= 0) {
    const int r = __popcll(m.who & ((uint64_t(1) << lane) - 1));
    lds.row[r] = lane * g.top_k + m.place;
  }
  __syncthreads();
  buf_t parts[kHParts];
  part_buffers<kHParts>(parts, o.h, g.T * g.top_k, Ip);
  HeldSweep<kHParts, G> sweep;
  for (int r0 = 0; r0 < members; r0 += G * RG) {
    if (r0 > 0) __syncthreads();
    const int rows = min(members - r0, G * RG), groups = (rows + RG - 1) / RG;
    hold_rows<kHParts>(lds, parts, rows, ld, c0, chunks, blocks, wave, lane,
                  [&](int r) { return 2 * Ip * __builtin_amdgcn_readfirstlane(lds.row[r0 + r]); },
                  [&] { sweep.begin(tile + wave, tiles, chunks, fetch); });
    sweep.run(lds.rows, ld, groups, tiles, chunks, lane, fetch, [&](int t, const f32x4_t (&acc)[G][2]) {
#pragma unroll
      for (int i = 0; i < G; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int rr = held_row<kHParts>(quad, q), r = RG * i + rr;
          if (rr >= RG || r >= rows) continue;
          float* z = o.z + ((int64_t)blockIdx.z * g.T * g.top_k + lds.row[r0 + r]) * Dz + 32 * t + l16;
          z[0] = acc[i][0][q], z[16] = acc[i][1][q];
        }
    });
  }
}

// The same for up to 4 tokens and 64 choices whose h fits LDS, at once or in two turns: a workgroup has 16 columns of y
// whole, its 16 waves taking chunks of all chosen experts in turn; nothing is left to add across workgroups (one token, 8 of
// 128 experts of 2048 x 768: 7.0 us, by the kernel before 8.7).
constexpr int kFewWaves = 16, kFewLds = 140 << 10;

// `range` chunks of a row are in LDS at once: all, or (TWICE) half of them.
template <bool TWICE>
__global__ __launch_bounds__(64 * kFewWaves) void moe_down_few_kernel(MoeArgs g, MoeBufs o, int range, uint32_t inverse,
                                                                      int step_x, int step_c) {
  __shared__ __align__(16) char hs[kFewLds];  // h's rows, of each its parts, chunks kRowBytes apart
  __shared__ float sums[kFewWaves][16][17];
  const int lane = threadIdx.x & 63, k = g.top_k, places = g.T * k;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  static_assert(kHParts <= 4, "a row's parts are rows of the product");
  const int l16 = lane & 15, quad = lane >> 4, strip = (int)blockIdx.x;
  const int chunks = mx4_chunks(g.I), blocks = mx4_blocks(g.I);
  const int id = lane < places ? o.ids[lane] : -1;
  // h to LDS, a chunk of a row's part a turn (what lies past a row's last chunk counts for nothing)
  constexpr int HELD = 4;
  const int turns = places * kHParts * range;
  u32x4_t v[HELD];
  auto get = [&](int t, int c0) {
    int at = t;
    if (TWICE) {
      const int row = (int)((uint32_t)t * inverse >> 16);
      at = row * chunks + min(c0 + t - row * range, chunks - 1);
    }
    return *reinterpret_cast<const u32x4_t*>(o.h + (int64_t)512 * at + 8 * lane);
  };
  auto put = [&](int t, const u32x4_t& x) { *reinterpret_cast<u32x4_t*>(hs + t * kRowBytes + 16 * lane) = x; };
  auto first_turns = [&](int c0) {
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (wave + i * kFewWaves < turns) v[i] = get(wave + i * kFewWaves, c0);
  };
  first_turns(0);
  __builtin_amdgcn_sched_barrier(0);
  // the places whose expert no earlier one has
  bool first = id >= 0;
  for (int p = 0; p + 1 < places; ++p) first = first && !(p < lane && __builtin_amdgcn_readlane(id, p) == id);
  const uint64_t firsts = __ballot(first);
  const int rank = __popcll(firsts & ((uint64_t(1) << lane) - 1)), experts = __popcll(firsts);
  // A wave's units: chunk c0 + c of the x-th chosen expert, the kFewWaves-th next one each time, of the chunks from c0 on that are
  // in LDS.  (Without divisions: step_x and step_c are kFewWaves over range, and its remainder.)
  struct Unit {
    int x, c, c0;
  };
  auto after = [&](const Unit& u) {
    Unit n = {u.x + step_x, u.c + step_c, u.c0};
    if (n.c >= range) n.c -= range, ++n.x;
    return n;
  };
  auto expert = [&](const Unit& u) {
    return __builtin_amdgcn_readlane(id, (int)__builtin_ctzll(__ballot(first && rank == u.x) | (uint64_t(1) << 63)));
  };
  auto request = [&](MoeChunk& w, const Unit& u) {
    const uint8_t* p = nullptr;
    if (u.x < experts && (!TWICE || u.c0 + u.c < chunks))
      p = g.wd + (int64_t)expert(u) * mx4_weight_bytes(g.D, g.I) + (int64_t)strip * mx4_strip_bytes(g.I) +
          (int64_t)kChunkBytes * (u.c0 + u.c);
    load_chunk(w, p, blocks - 16 * (u.c0 + u.c), lane);
  };
  MoeChunk w[2];
  Unit begin, u0, u1;
  begin.x = (int)((uint32_t)wave * inverse >> 16), begin.c = wave - begin.x * range, begin.c0 = 0;
  u0 = begin, u1 = after(u0);
  request(w[0], u0);
  request(w[1], u1);
  __builtin_amdgcn_sched_barrier(0);
  auto rest = [&](int c0) {
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (wave + i * kFewWaves < turns) put(wave + i * kFewWaves, v[i]);
    for (int t = wave + HELD * kFewWaves; t < turns; t += kFewWaves) put(t, get(t, c0));
    __syncthreads();
  };
  rest(0);

  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  auto use = [&](const MoeChunk& m, const Unit& u) {
    const int e = expert(u);
    // row l16 is part l16 / 4 of token l16 % 4, its first place with this expert
    const uint64_t same = __ballot(id == e);
    const int token = l16 % 4, part = l16 / 4;
    const uint32_t own = token < g.T && part < kHParts ? (uint32_t)(same >> (token * k)) & (uint32_t)((uint64_t(1) << k) - 1) : 0u;
    const int row = own == 0 ? 0 : part * places + token * k + __builtin_ctz(own);
    const char* from = own == 0 ? hs : hs + (row * range + u.c) * kRowBytes + 16 * quad;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool ok = own != 0 && 4 * quad + j < blocks - 16 * (u.c0 + u.c);
      const float sc = scale_f32((m.s >> (8 * j)) & 255);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bf16x8_t b = __builtin_bit_cast(bf16x8_t, bf16_of_codes(m.c[j][i], sc));
        u32x4_t a = *reinterpret_cast<const u32x4_t*>(from + (ok ? 256 * j + 64 * i : 0));
        if (!ok) a = u32x4_t{0u, 0u, 0u, 0u};
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), b, acc, 0, 0, 0);
      }
    }
  };
  // pairs of units, the next pair's weights on their way; after the last of some chunks the first of the next
  for (;;) {
    Unit n0 = after(u1);
    const bool end = n0.x >= experts;
    if (TWICE && end) n0 = begin, n0.c0 = u0.c0 + range;
    const Unit n1 = after(n0);
    if (u0.x < experts) use(w[0], u0);
    request(w[0], n0);
    if (u1.x < experts) use(w[1], u1);
    request(w[1], n1);
    if (end) {
      if (!TWICE || n0.c0 >= chunks) break;
      first_turns(n0.c0);
      __syncthreads();
      rest(n0.c0);
    }
    u0 = n0, u1 = n1;
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) sums[wave][4 * quad + r][l16] = acc[r];
  __syncthreads();
  const int m = threadIdx.x / 16, n = 16 * strip + (int)threadIdx.x % 16;
  if (m >= g.T || n >= g.D) return;
  float y = 0.f;
#pragma unroll
  for (int i = kHParts; i-- > 0;)
#pragma unroll
    for (int q = 0; q < kFewWaves; ++q) y += sums[q][4 * i + m][threadIdx.x % 16];
  with_y(g.y, g.y_dtype, [&](auto* yt) {
    typedef typename std::remove_pointer<decltype(yt)>::type Y;
    yt[(int64_t)m * g.ldy + n] = (Y)y;
  });
}

// A token's sums by a launch of its own, a workgroup for 256 columns.
__global__ __launch_bounds__(256) void moe_join_kernel(MoeArgs g, MoeBufs o, int Dz, int blocks, int ranges) {
  const int t = (int)blockIdx.x / blocks, n = ((int)blockIdx.x % blocks) * 256 + (int)threadIdx.x, k = g.top_k;
  const buf_t zb = make_buf(o.z, 4u * (uint32_t)(g.T * k) * (uint32_t)Dz * (uint32_t)ranges);
  // the places whose expert no earlier one has
  const int lane = threadIdx.x & 63, id = lane < k ? o.ids[t * k + lane] : -1;
  bool first = id >= 0;
  for (int p = 0; p + 1 < k; ++p) first = first && !(p < lane && __builtin_amdgcn_readlane(id, p) == id);
  const uint32_t firsts = (uint32_t)__ballot(first);
  if (n >= g.D) return;
  const float v = token_sum<false>(zb, t * k, k, Dz, n, ranges, g.T * k, [&](int p) { return (firsts >> p) & 1; });
  with_y(g.y, g.y_dtype, [&](auto* yt) {
    typedef typename std::remove_pointer<decltype(yt)>::type Y;
    yt[(int64_t)t * g.ldy + n] = (Y)v;
  });
}

// ---------------------------------------------------------------- host side
// Whether workgroups, one on each CU, hold an expert's rows, and of how many row groups: 0 not.  `split`: whether they may
// hold a range of a row's chunks; `least`: tiles that each has, else not.  Taken for what tokens that choose evenly would
// choose: groups for all but a few experts' rows, and more where they cost no further range (an expert with more rows has
// its weights read again for each so many).
template <int P> static HeldPlan plan_held(int T, int top_k, int E, int chunks, bool split, int tiles, int least) {
  constexpr int RG = kHeldRows<P>, MOST = kHeldGroups<P>;
  float none = 1.f;  // (given experts may be more than there are)
  for (int t = 0; t < T; ++t) none *= 1.f - (float)(top_k < E ? top_k : E) / (float)E;
  const float chosen = (float)E * (1.f - none), mean = (float)(T * top_k) / chosen;
  HeldPlan p{};
  const float rows = fminf((float)T, mean + 2.f * sqrtf(mean));
  p.groups = 1;
  while (p.groups < MOST && rows > (float)(RG * p.groups)) ++p.groups;
  while (p.groups < MOST && T > RG * p.groups && chunks <= held_chunks<P>(p.groups + 1)) ++p.groups;
  const int most = held_chunks<P>(p.groups);
  p.ranges = (chunks + most - 1) / most;
  if (p.ranges > 1 && !split) return HeldPlan{};
  p.range = (chunks + p.ranges - 1) / p.ranges;
  p.ranges = (chunks + p.range - 1) / p.range;
  const float parts = chosen * (float)p.ranges;
  const int wgs = parts < 256.f ? (int)(256.f / parts) : 1;
  p.per = (tiles + wgs - 1) / wgs;
  return p.per < least ? HeldPlan{} : p;
}

MoePlan plan_moe(int T, int D, int I, int E, int top_k, int x_dtype) {
  MoePlan p{};
  p.xparts = x_dtype == YF32 ? 3 : x_dtype == XF16 ? 2 : 1;
  p.Dp = (int)round_up(D, 512);
  p.Ip = (int)round_up(I, 512);
  p.Dz = (int)round_up(D, 32);
  // (held in LDS or not, 18 tiles a workgroup: 45 and 39 us; 22 tiles: 41 and 48)
  const auto plan_up = p.xparts == 1 ? plan_held<1> : p.xparts == 2 ? plan_held<2> : plan_held<3>;
  p.up = plan_up(T, top_k, E, mx4_chunks(D), false, 2 * mx4_blocks(I), 20);
  // (64 tokens; held in LDS or not, 10 tiles a workgroup: 26 and 31 us; 16 tiles: 34 and 44; 22 tiles: 39 and 56.  16 tokens,
  // 13 tiles, where the additions then take a launch more: 79 and 79 for all)
  p.down = plan_held<kHParts>(T, top_k, E, mx4_chunks(I), true, p.Dz / 32, 10);
  const int64_t z = (int64_t)T * top_k * p.Dz * 4;
  if (p.down.ranges > 1 && z * p.down.ranges > kRangesBytes) p.down = HeldPlan{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (size_t)round_up((int64_t)bytes, 256);
    return o;
  };
  p.ids = take((size_t)T * top_k * 4);
  p.w = take((size_t)T * top_k * 4);
  p.done = take((size_t)p.Dz / 32 * 4);
  p.x = take((size_t)p.xparts * T * p.Dp * 2);
  p.h = take((size_t)kHParts * T * top_k * p.Ip * 2);
  p.z = take((size_t)z * (p.down.ranges > 1 ? p.down.ranges : 1));
  p.bytes = at;
  return p;
}

template <int XP> static hipError_t moe_t(const MoeArgs& a, const MoePlan& p, const MoeBufs& o, hipStream_t s) {
  // a workgroup for each expert, or for each place of the tokens' choices if these are fewer; of more tiles than
  // about 3 rounds of workgroups (2 on a CU) would be, a workgroup takes several in turn
  const int pairs = a.T * a.top_k < a.E, slots = pairs ? a.T * a.top_k : a.E;
  auto each = [&](int tiles) { return (int)(((int64_t)tiles * slots + 1535) / 1536); };
  const int up = 2 * mx4_blocks(a.I), down = p.Dz / 32, per_up = each(up), per_down = each(down);
  const int xg = (a.T * (p.Dp / 8) + 255) / 256, gd = (down + per_down - 1) / per_down;
  // where every workgroup makes the choices, all are on the chip at once (4 tokens, 8 of 128 experts of 2048 x 768: 31.4 us, in
  // three rounds 36.5)
  const int per_few = (int)(((int64_t)up * slots + 511) / 512);
  hipError_t e = hipSuccess;
  if (a.T <= 4) {
    constexpr int XT = kTypeOfParts<XP>;
    const bool vec = vec8_ok(a.x, a.ldx, a.D, a.x_dtype == YF32 ? 4 : 2) && a.D % 8 == 0;
    e = launch_kernel(vec ? moe_up_few_kernel<XT, XP, true> : moe_up_few_kernel<XT, XP, false>, dim3((unsigned)((up + per_few - 1) / per_few), (unsigned)slots),
                      dim3(64 * kMoeWaves), s, a, o, p.Ip, pairs, per_few, gd);
  } else {
    e = launch_kernel(moe_route_kernel<XP>, dim3((unsigned)((a.T + 3) / 4 + (xg < 256 ? xg : 256))), dim3(256), s, a, o, gd, p.Dp);
    if (e != hipSuccess) return e;
    const HeldPlan& held = p.up;
    if (held.groups != 0) {
      e = launch_kernel(held.groups == 1   ? moe_up_held_kernel<XP, 1>
                        : held.groups == 2 ? moe_up_held_kernel<XP, 2>
                                           : moe_up_held_kernel<XP, kHeldGroups<XP>>,
                        dim3((unsigned)((up + held.per - 1) / held.per), (unsigned)slots), dim3(64 * kHeldWaves), s, a, o, p.Dp,
                        p.Ip, pairs, held.per);
    } else {
      e = launch_kernel(a.T <= kRowGroup<XP> ? moe_up_kernel<XP, 1> : moe_up_kernel<XP, 2>,
                        dim3((unsigned)((up + per_up - 1) / per_up), (unsigned)slots), dim3(64 * kMoeWaves), s, a, o, p.Dp, p.Ip,
                        pairs, per_up);
    }
  }
  if (e != hipSuccess) return e;
  const int places = a.T * a.top_k;
  const int chunks = mx4_chunks(a.I);
  // (in two turns and by the other kernels, us: 3 tokens, 8 of 128 experts of 2048 x 768, 26.6 and 30.6; 4 tokens 31.1 and
  // 30.7; one token, 2 of 8 experts of 4096 x 14336, 41.3 and 42.0)
  auto fits = [&](int range) { return (int64_t)places * kHParts * range * kRowBytes <= kFewLds; };
  const int range = fits(chunks) ? chunks : (chunks + 1) / 2;
  if (a.T <= 4 && places <= 64 && fits(range))
    return launch_kernel(range == chunks ? moe_down_few_kernel<false> : moe_down_few_kernel<true>, dim3((unsigned)((a.D + 15) / 16)), dim3(64 * kFewWaves), s, a, o, range,
                         (uint32_t)((65536 + range - 1) / range), kFewWaves / range, kFewWaves % range);
  const HeldPlan& held = p.down;
  const bool join = held.groups == 0 && a.T <= 16;
  if (held.groups != 0)
    e = launch_kernel(held.groups == 1   ? moe_down_held_kernel<1>
                      : held.groups == 2 ? moe_down_held_kernel<2>
                                         : moe_down_held_kernel<kHeldGroups<kHParts>>,
                      dim3((unsigned)((down + held.per - 1) / held.per), (unsigned)slots, (unsigned)held.ranges), dim3(64 * kHeldWaves), s, a,
                      o, p.Ip, pairs, p.Dz, held.per, held.range);
  else
    e = launch_kernel(!join ? moe_down_kernel<2, false>
                            : a.T <= kRowGroup<kHParts> ? moe_down_kernel<1, true> : moe_down_kernel<2, true>,
                      dim3((unsigned)gd, (unsigned)slots), dim3(64 * kMoeWaves), s, a, o, p.Ip, pairs, p.Dz, per_down);
  if (e != hipSuccess || join) return e;
  const int columns = (a.D + 255) / 256;
  return launch_kernel(moe_join_kernel, dim3((unsigned)(a.T * columns)), dim3(256), s, a, o, p.Dz, columns,
                       held.groups != 0 ? held.ranges : 1);
}


hipError_t launch_mx4_moe(const MoeArgs& a, const MoePlan& p, hipStream_t s) {
  char* ws = static_cast<char*>(a.ws);
  MoeBufs o{};
  o.ids = reinterpret_cast<int*>(ws + p.ids);
  o.w = reinterpret_cast<float*>(ws + p.w);
  o.done = reinterpret_cast<uint32_t*>(ws + p.done);
  o.x = reinterpret_cast<uint16_t*>(ws + p.x);
  o.h = reinterpret_cast<uint16_t*>(ws + p.h);
  o.z = reinterpret_cast<float*>(ws + p.z);
  switch (p.xparts) {
    case 1: return moe_t<1>(a, p, o, s);
    case 2: return moe_t<2>(a, p, o, s);
  }
  return moe_t<3>(a, p, o, s);
}

}  // namespace qmm
