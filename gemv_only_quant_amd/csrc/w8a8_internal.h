// w8a8_internal.h -- launchers of the int8 x int8 operators (not public).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "qmm_internal.h"

namespace qmm {

// Data types as in qmm.h / qmm_int8.h: 0 fp16, 1 bf16, 2 fp32, 3 int8.
constexpr int kTypeI8 = 3;
enum { ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2 };

__host__ __device__ constexpr int64_t round_up(int64_t v, int64_t to) {
  return (v + to - 1) / to * to;
}

// Bytes of contraction per stage of the tile kernels: operands that the library
// lays out itself are zero-padded to whole stages.
constexpr int kStageBytes = 128;
// Columns of the gradients' operands that share a level (fp16): of d and of dt.
constexpr int kLevelD = 32, kLevelT = 16;

// A launch has at most 2^32 - 1 threads (of a larger grid the rest is dropped without an
// error): workgroups of 256 threads of one launch, and rows that a launch is given.
constexpr int64_t kMaxGroups = (int64_t(1) << 24) - 1;
constexpr int kMaxLaunchRows = 1 << 22;

// ---- per-token quantizer (w8a8_quantize.hip) -------------------------------
hipError_t launch_quantize_tokens(const void* x, int x_dtype, int64_t ldx, int8_t* xq,
                                  int64_t ldxq, float* sx, int M, int K, hipStream_t s);

// ---- products of codes, forward --------------------------------------------
struct W8A8Args {
  const int8_t* x;
  int64_t ldx;
  const float* sx;
  const int8_t* w[2];  // w[1]: the up projection (gated only)
  const float* sw[2];
  int64_t ldw;
  void* y;
  int y_dtype;
  int64_t ldy;
  int M, N, K;
  bool gated;
  int act;
  hipStream_t stream;
};
hipError_t launch_w8a8(const W8A8Args& a);
// A few tokens (w8a8_rows.hip): x of any type, quantized within the launch
// where it is not codes (a.x and a.sx then count for nothing).
bool rows_fits(int M, int K);
// The tokens' codes lie in LDS in rows of ldk bytes, and step u of a wave's batch starts
// at byte k of them.  Whether the row has it: a batch's later steps may lie past its end,
// and of SHARED waves on a column those without a batch have no step at all.
template <int SHARED> __host__ __device__ constexpr bool rows_step_exists(int k, int u, int ldk) {
  return (SHARED == 1 && u == 0) || k < ldk;
}
hipError_t launch_rows(const W8A8Args& a, const void* x, int x_dtype, int64_t ldx);

// ---- gradients -------------------------------------------------------------
// What a backward pass keeps in its workspace; offsets in bytes.
//   d      (M, Jp) dy sw (gated: dg sg | du su), Jp = parts * Np
//   dt     (parts * Nr, Mp) dy sx transposed (rows N .. Nr of a part unused)
//   de, dte  fp16: the level of each kLevelD columns of d (one for all parts: (M, Np /
//          kLevelD) bytes) and of each kLevelT columns of dt ((parts * Nr, Mp / kLevelT))
//   inv, invt  fp16: what the products' rows are multiplied by, (M) and (parts * Nr)
//   part   fp32 shares of dx's product or dW's, where K is split
// with the contracted axes zero-padded to whole stages.
// How launch_tile_plain makes a product: tiles of 32 w (8 or 4), the contraction in
// `splits` shares (1: whole; more with w = 4 alone).
struct PlainPlan {
  int w, splits;
};
PlainPlan plain_plan(int64_t M, int64_t N, int64_t kb);

struct BackwardPlan {
  int parts;
  int64_t Np, Jp, Nr, Mp;
  size_t d, dt, de, dte, inv, invt, part, bytes;
  PlainPlan dx, dw;
};
BackwardPlan plan_backward(int M, int N, int K, bool gated, bool weight_grad);

struct BackwardArgs {
  const void* dy;
  int dtype;  // XF16 / XBF16
  int64_t lddy;
  const int8_t* x;
  int64_t ldx;
  const float* sx;
  const int8_t* w[2];
  const float* sw[2];
  int64_t ldw;
  void* dx;
  int64_t lddx;
  void* dw[2];
  int64_t lddw;
  int M, N, K;
  bool gated;
  int act;
  void* ws;
  hipStream_t stream;
};
hipError_t launch_backward(const BackwardArgs& a, const BackwardPlan& p);

// Zeros a (rows, cols) matrix of elements of `size` bytes (empty sums).
hipError_t launch_fill_zero(void* y, int size, int64_t ld, int rows, int cols, hipStream_t s);

// ---- tile kernels (w8a8_large.hip) ------------------------------------------
// C (rows M of A, rows N of B) = A B^t over `kb` contracted bytes of A; element
// types and what becomes of C are the kernel's.
struct TileArgs {
  const void* a;       // (M, kb bytes), leading dimension lda bytes
  int64_t lda;
  const void* b[2];    // int8: (N, kb bytes) each.  16-bit: codes (brows, N) each, the
  int64_t ldb;         // contracted axis their rows, each padded to bpad of it
  int brows, bpad;
  int M, N, kb;
  const float* sa;     // scale of each row of A (int8), factor of each row of C (plain, fp16)
  const float* sb[2];  // scale of each row of B (int8)
  void* y;
  int y_dtype;
  int64_t ldy;
  void* y2;            // plain: where rows M2 and up go (as rows 0 and up)
  int M2, Mv;          // plain: rows of one output, and how many of them exist
  int act;
  // gradient of the gated block (int8 products with a gradient epilogue)
  const void* dh;
  int64_t lddh;
  void* d;             // (M, 2 Np)
  void* dt;            // (2 Nr, Mp) or NULL
  uint8_t *de, *dte;   // their levels (fp16)
  int64_t Np, Nr, Mp;
  // plain: the shares' fp32 sums, where K is split, lie in part (splits, M, N rounded
  // up to 4) and are added in a fixed order by a second launch
  PlainPlan plan;
  float* part;
};
hipError_t launch_tile_scale(const TileArgs& t, hipStream_t s);
hipError_t launch_tile_gated(const TileArgs& t, hipStream_t s);
hipError_t launch_tile_grad(const TileArgs& t, int dtype, hipStream_t s);
hipError_t launch_tile_plain(const TileArgs& t, int dtype, hipStream_t s);
// A decode batch (w8a8_skinny.hip).
bool skinny_fits(int M);
hipError_t launch_skinny(const TileArgs& t, bool gated, hipStream_t s);
}  // namespace qmm
