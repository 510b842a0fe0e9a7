/*
 * qmm_int8.h -- int8 x int8 products with a scale for each token and each
 * output channel, the gated feed-forward block on them, and their gradients,
 * for AMD Instinct MI355X (gfx950).  Part of libqmm.so; status codes, error
 * text and data types are qmm.h's.
 *
 *   quantizer  sx[m] = max_k |x[m][k]| / 127,  xq[m][k] = rint(x[m][k] / sx[m])
 *   product    y[m][n] = sx[m] sw[n] sum_k xq[m][k] W[n][k]
 *   gated      h[m][n] = act(g[m][n]) u[m][n],  g and u products with Wg and Wu
 *   gradients with respect to the values x^ = sx xq and W^ = sw W (what a
 *   straight-through estimator passes on to the values that were quantized):
 *     product  dx = dy W^,              dW = dy^t x^
 *     gated    dg = dh u act'(g), du = dh act(g),
 *              dx = dg Wg^ + du Wu^,    dWg = dg^t x^,  dWu = du^t x^
 *
 * The int8 weights (N, K) with an fp32 scale for each row are tiny-llm's
 * (src/tinyllm/kernels/int8_gemv.py, int8_matmul), as qmm_gemv takes them;
 * what is added is the 8-bit left operand.
 *
 * Conventions
 *  - Pointers are device pointers, `stream` is a hipStream_t.  Calls are
 *    asynchronous on it, never synchronise and never allocate.  Every
 *    argument is checked before any HIP call.
 *  - A matrix is row-major with a leading dimension ld* in elements, at
 *    least its row length (at least 1).  int8 matrices start on 16 bytes
 *    and have a leading dimension that is a multiple of 16; K itself may be
 *    anything.  Where K % 16 != 0 the bytes that follow a row up to the next
 *    multiple of 16 are read (the last row's too) and take no part in the
 *    result, whatever they hold.  Other matrices need the alignment of their
 *    elements only; 16-byte aligned ones with rows of whole 16 bytes run
 *    faster.
 *  - Leading dimensions stay below 2^22 elements (2^22 bytes for int8), K
 *    below 2^17: sums of K products of codes then fit 32 bits and are exact
 *    whole numbers, whatever the order; M and N at most 2^31 - 1025, in the
 *    backward calls M, N (gated: 2 N) below 2^21 - 256 (QMM_ERR_UNSUPPORTED
 *    beyond).
 *  - Outputs are fully overwritten (the elements of their rows; nothing
 *    between rows is touched) and must not overlap inputs.  An empty sum is
 *    zero: K == 0 writes y = 0, M == 0 writes dW = 0, N == 0 writes dx = 0.
 *    A call without outputs is a no-op.
 *  - Results are the same from run to run, bit for bit.
 */
#ifndef QMM_INT8_H
#define QMM_INT8_H

#include "qmm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* x_dtype of activations that are codes already (with their scales in sx) */
#define QMM_I8 3

typedef enum {
    QMM_SILU = 0,      /* v / (1 + exp(-v)) */
    QMM_GELU = 1,      /* v / 2 (1 + erf(v / sqrt 2)) */
    QMM_GELU_TANH = 2  /* v / 2 (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3))) */
} qmm_act;

/*
 * qmm_quantize_tokens: x (M, K) of x_dtype (QMM_F32, QMM_F16, QMM_BF16) to
 * codes xq (M, K) int8 in [-127, 127] and scales sx (M,) fp32.
 *   sx = max |x| / 127 rounded to fp32; a code is the exact quotient x / sx
 *   rounded to nearest even (and clamped, which matters only where sx is
 *   subnormal).  A row of zeros has scale 0 and codes 0.  A row that holds
 *   an infinity or a NaN has scale NaN and codes 0: all of its outputs are
 *   NaN, and no other row's are.
 * The bytes of a row of xq from K up to the next multiple of 16 are set to 0
 * (so ldxq must reach there).
 */
QMM_API qmm_status qmm_quantize_tokens(const void* x, int x_dtype, int64_t ldx, int8_t* xq,
                                       int64_t ldxq, float* sx, int M, int K, void* stream);

/* Scratch for activations that the call quantizes itself (x_dtype other than
 * QMM_I8): codes and scales.  Device memory, 16-byte aligned, any contents;
 * in use until the call's work on the stream is done.  0 for QMM_I8, for a few
 * tokens (which are quantized within the product's launch) and for invalid
 * arguments. */
QMM_API size_t qmm_w8a8_workspace_bytes(int M, int K, int x_dtype);

/*
 * qmm_w8a8_gemm: y (M, N) of y_dtype (QMM_F32, QMM_F16, QMM_BF16).
 * x is either codes with their scales (x_dtype QMM_I8, sx not NULL) or values
 * (sx NULL), which the call quantizes as qmm_quantize_tokens does.  The whole
 * sum is exact; it is rounded to fp32 once, multiplied by sx[m] sw[n] in
 * fp32 and rounded to y's type.
 */
QMM_API qmm_status qmm_w8a8_gemm(const void* x, int x_dtype, int64_t ldx, const float* sx,
                                 const int8_t* W, int64_t ldw, const float* sw, void* y,
                                 int y_dtype, int64_t ldy, int M, int N, int K, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* qmm_w8a8_gated: h (M, N) = act(x^ Wg^t) * (x^ Wu^t), both products, the
 * activation and the product in one pass, in fp32, rounded once to h's type.
 * x as for qmm_w8a8_gemm; Wg and Wu (N, K) have the leading dimension ldw. */
QMM_API qmm_status qmm_w8a8_gated(const void* x, int x_dtype, int64_t ldx, const float* sx,
                                  const int8_t* Wg, const float* sg, const int8_t* Wu,
                                  const float* su, int64_t ldw, void* h, int h_dtype, int64_t ldh,
                                  int M, int N, int K, int act, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* Scratch of a backward call (gated: 0 or 1; weight_grad: 0 or 1).  Device
 * memory, 256-byte aligned, any contents.  0 for invalid arguments. */
QMM_API size_t qmm_w8a8_backward_workspace_bytes(int M, int N, int K, int gated, int weight_grad);

/*
 * qmm_w8a8_gemm_backward: dx (M, K) and, where dW is not NULL, dW (N, K),
 * both of dy's type (QMM_F16 or QMM_BF16).  dx[m][k] = sum_n dy[m][n] sw[n]
 * W[n][k]; dW[n][k] = sum_m dy[m][n] sx[m] xq[m][k].  Products are formed on
 * the matrix cores from operands of dy's type (the codes are exact in it;
 * dy sw and dy sx are each rounded to it once), summed in fp32 and rounded once.
 * In fp16 each token's dy sw, and each channel's dy sx, has a power of two of its
 * own, taken out of its sums again: none leaves the range, and next to a row's
 * largest value the others lose less than 2^-30 of it beside their rounding.  sx
 * and xq are read for dW alone and may be NULL without it.
 */
QMM_API qmm_status qmm_w8a8_gemm_backward(const void* dy, int dtype, int64_t lddy,
                                          const int8_t* xq, int64_t ldx, const float* sx,
                                          const int8_t* W, int64_t ldw, const float* sw, void* dx,
                                          int64_t lddx, void* dW, int64_t lddw, int M, int N,
                                          int K, void* workspace, size_t workspace_bytes,
                                          void* stream);

/*
 * qmm_w8a8_gated_backward: dx (M, K) and, where dWg and dWu are not NULL
 * (both or neither), dWg and dWu (N, K), all of dh's type.  g and u are made
 * again from the codes (exact sums, fp32), so the forward pass keeps nothing
 * of size M x N.  dg and du are formed in fp32; dg sg, du su, dg sx and du sx
 * are rounded to dh's type as above (dg sg and du su of a token share its power of
 * two), so dg and du themselves may lie beyond fp16's range.
 */
QMM_API qmm_status qmm_w8a8_gated_backward(const void* dh, int dtype, int64_t lddh,
                                           const int8_t* xq, int64_t ldx, const float* sx,
                                           const int8_t* Wg, const float* sg, const int8_t* Wu,
                                           const float* su, int64_t ldw, void* dx, int64_t lddx,
                                           void* dWg, void* dWu, int64_t lddw, int M, int N, int K,
                                           int act, void* workspace, size_t workspace_bytes,
                                           void* stream);

#ifdef __cplusplus
}
#endif
#endif /* QMM_INT8_H */
