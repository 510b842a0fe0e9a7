// mx4_internal.h -- launchers of the microscaled 4-bit operators (not public).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "w8a8_internal.h"

namespace qmm {

// Data types as in qmm.h / qmm_int8.h / qmm_mx4.h: 0 fp16, 1 bf16, 2 fp32, 4 mx4.

// ---- layouts ---------------------------------------------------------------
constexpr int kBlock = 32;  // values that share a scale
__host__ __device__ constexpr int mx4_blocks(int K) { return (K + kBlock - 1) / kBlock; }
// packed weights: chunks of 512 values of strips of 16 columns
constexpr int kChunkBytes = 4096 + 256;
__host__ __device__ constexpr int mx4_chunks(int K) { return (K + 511) / 512; }
__host__ __device__ constexpr int64_t mx4_strip_bytes(int K) { return (int64_t)kChunkBytes * mx4_chunks(K); }
__host__ __device__ constexpr int64_t mx4_weight_bytes(int N, int K) {
  return (int64_t)((N + 15) / 16) * mx4_strip_bytes(K);
}

// ---- quantizer, its inverse, packing (mx4_quantize.hip) ---------------------
hipError_t launch_mx4_quantize(const void* x, int x_dtype, int64_t ldx, uint8_t* codes, int64_t ldc,
                               uint8_t* scales, int64_t lds, int M, int K, hipStream_t s);
hipError_t launch_mx4_dequantize(const uint8_t* codes, int64_t ldc, const uint8_t* scales,
                                 int64_t lds, void* y, int y_dtype, int64_t ldy, int M, int K,
                                 hipStream_t s);
hipError_t launch_mx4_pack(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds,
                           void* W, int batch, int N, int K, hipStream_t s);

// Values straight to the packed layout of a weight (M, K).  (Rows past M of the last strip: anything.)
hipError_t launch_mx4_quantize_packed(const void* x, int x_dtype, int64_t ldx, uint8_t* w, int M, int K,
                                      hipStream_t s);

// ---- product ---------------------------------------------------------------
struct Mx4Args {
  const uint8_t* a;  // packed (M, K)
  const uint8_t* w;  // packed (N, K)
  void* y;
  int y_dtype;
  int64_t ldy;
  int M, N, K;
};
// Few values (mx4_skinny.hip): quantized within the launch; a.a counts for nothing.
bool mx4_rows_fits(int M, int K);
hipError_t launch_mx4_rows(const Mx4Args& a, const void* x, int x_dtype, int64_t ldx, hipStream_t s);
// Up to 64 rows or some more, and many (mx4_large.hip).
bool mx4_skinny_fits(int M, int N);
hipError_t launch_mx4_skinny(const Mx4Args& a, hipStream_t s);
hipError_t launch_mx4_large(const Mx4Args& a, hipStream_t s);

// ---- mixture of experts (mx4_moe.hip) ---------------------------------------
constexpr int kMoeTokens = 64, kMoeTopK = 32, kMoeExperts = 1024;
struct MoeArgs {
  const void* x;
  int x_dtype;
  int64_t ldx;
  const uint8_t *wg, *wu, *wd;
  void* y;
  int y_dtype;
  int64_t ldy;
  int T, D, I, E, top_k, act;
  const void* logits;  // or NULL
  int logits_dtype;
  int64_t ldl;
  int renormalize;
  const void* ids;
  int ids_size;
  const void* weights;
  int weights_dtype;
  void* ws;
};
// What a call keeps in its workspace (offsets in bytes; MoeBufs in mx4_moe.hip): the choices, counters, x and h as
// sums of bf16 parts in rows padded to whole blocks, the experts' rows of y in whole strips.
struct HeldPlan {
  int groups, range, ranges, per;  // row groups in LDS (0: none), chunks of a row there, ranges of these; tiles of a workgroup
};
struct MoePlan {
  int xparts;
  HeldPlan up, down;
  int Dp, Ip, Dz;
  size_t ids, w, done, x, h, z, bytes;
};
MoePlan plan_moe(int T, int D, int I, int E, int top_k, int x_dtype);
hipError_t launch_mx4_moe(const MoeArgs& a, const MoePlan& p, hipStream_t s);

}  // namespace qmm
