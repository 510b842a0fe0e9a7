// mx4_skinny.hip -- products of microscaled 4-bit codes, y = x^ W^t.
//
// A workgroup owns 16 rows and one strip of 16 columns; its 4 waves take steps
// of 128 values (a quarter of a chunk) in turn and add their sums in LDS.  The packed strip is the
// matrix cores' operand: 1 KiB of consecutive bytes per step.
#include "mx4_device.h"

namespace qmm {

__global__ __launch_bounds__(256) void mx4_skinny_kernel(Mx4Args g, int strips) {
  __shared__ float sums[4][16][17];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, quad = lane >> 4;
  const int strip = (int)(blockIdx.x % (unsigned)strips), m0 = 16 * (int)(blockIdx.x / (unsigned)strips);
  const int steps = 4 * mx4_chunks(g.K), blocks = mx4_blocks(g.K);
  const uint8_t* w = g.w + (int64_t)strip * mx4_strip_bytes(g.K);
  const int m = m0 + l16;
  const uint8_t* a = g.a + (int64_t)(m < g.M ? m : 0) * g.lda;
  const uint8_t* sa = g.sa + (int64_t)(m < g.M ? m : 0) * g.ldsa;
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  for (int s = wave; s < steps; s += 4) {
    const int b = 16 * (s / 4) + 4 * quad + s % 4;
    const uint8_t* c = w + (int64_t)kChunkBytes * (s / 4);
    const u32x4_t cb = *reinterpret_cast<const u32x4_t*>(c + 1024 * (s % 4) + 16 * lane);
    const uint32_t eb = c[4096 + 4 * lane + s % 4];
    u32x4_t ca = {0u, 0u, 0u, 0u};
    uint32_t ea = 127;
    if (b < blocks && m < g.M) {
      ca = *reinterpret_cast<const u32x4_t*>(a + 16 * b);
      ea = sa[b];
    }
    acc = mfma_mx4(ca, cb, acc, ea, eb);
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) sums[wave][4 * quad + r][l16] = acc[r];
  __syncthreads();
  const int row = threadIdx.x / 16, col = threadIdx.x % 16;
  const int n = 16 * strip + col;
  if (m0 + row >= g.M || n >= g.N) return;
  const float v = (sums[0][row][col] + sums[1][row][col]) + (sums[2][row][col] + sums[3][row][col]);
  with_y(g.y, g.y_dtype, [&](auto* yt) {
    typedef typename std::remove_pointer<decltype(yt)>::type Y;
    yt[(int64_t)(m0 + row) * g.ldy + n] = (Y)v;
  });
}

// ---------------------------------------------------------------- host side
bool mx4_skinny_fits(int M) { return M <= 64; }

hipError_t launch_mx4_skinny(const Mx4Args& a, hipStream_t s) {
  const int strips = (a.N + 15) / 16;
  const int64_t tiles = ((int64_t)a.M + 15) / 16;
  const int64_t most = kMaxGroups / strips > 0 ? kMaxGroups / strips : 1;
  if (strips > kMaxGroups) return hipErrorInvalidValue;
  hipError_t e = hipSuccess;
  for (int64_t t = 0; t < tiles && e == hipSuccess; t += most) {
    Mx4Args g = a;
    g.a += 16 * t * a.lda;
    g.sa += 16 * t * a.ldsa;
    g.y = static_cast<char*>(a.y) + 16 * t * a.ldy * (a.y_dtype == YF32 ? 4 : 2);
    g.M = (int)(a.M - 16 * t < 16 * most ? a.M - 16 * t : 16 * most);
    const int64_t now = ((int64_t)g.M + 15) / 16;
    e = launch_kernel(mx4_skinny_kernel, dim3((unsigned)(now * strips)), dim3(256), s, g, strips);
  }
  return e;
}

}  // namespace qmm
