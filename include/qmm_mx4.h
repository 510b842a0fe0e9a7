/*
 * qmm_mx4.h -- microscaled 4-bit floating point (mx4) for AMD Instinct MI355X
 * (gfx950): quantizer and its inverse, product, and a mixture-of-experts layer
 * for a few tokens.  Part of libqmm.so; status codes, error text and data types
 * are qmm.h's, activations qmm_int8.h's.
 *
 *   a row's 32 consecutive values of a block share a scale X = 2^(e - 127), e a
 *   byte (255: not a number); a value is X times its code's value
 *   0 0.5 1 1.5 2 3 4 6 (codes 0 to 7; 8 to 15 their negatives)
 *   quantizer  e = floor(log2 max |x|) - 2 + 127, at least 0;
 *              code = x / X rounded to nearest even, held to +-6
 *   product    y[m][n] = sum_k x^[m][k] W[n][k]
 *   mixture    y[t] = sum_j w[t][j] Wd_e (act(Wg_e x[t]) * (Wu_e x[t])), e = ids[t][j]
 *
 * Conventions
 *  - Pointers are device pointers, `stream` is a hipStream_t.  Calls are
 *    asynchronous on it, never synchronise and never allocate.  Every
 *    argument is checked before any HIP call.
 *  - Codes lie two to a byte, the earlier one in the low half, in rows of whole
 *    blocks: a row of K values has B = ceil(K / 32) blocks, 16 B bytes of codes
 *    and B bytes of scales.  Codes past K count as values (the quantizer makes
 *    them zeros).  Matrices are row-major with a leading dimension ld* in
 *    elements (bytes, for codes and scales).
 *  - Other matrices need the alignment of their elements only; 16-byte aligned
 *    ones with rows of whole 16 bytes run faster.
 *  - Sizes: K, D and I below 2^20, leading dimensions below 2^22 elements (2^22
 *    bytes for codes and scales), M and N at most 2^31 - 1025
 *    (QMM_ERR_UNSUPPORTED beyond).
 *  - Outputs are fully overwritten (the elements of their rows; nothing between
 *    rows is touched but the padding of qmm_mx4_quantize's scales) and must not overlap inputs.  An empty sum is zero.  A
 *    call without outputs is a no-op.
 *  - Results are the same from run to run, bit for bit.
 */
#ifndef QMM_MX4_H
#define QMM_MX4_H

#include "qmm_int8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* x_dtype of activations that are mx4 codes already (with their scales in sx) */
#define QMM_MX4 4
/* most tokens and chosen experts of a token, most experts of qmm_mx4_moe */
#define QMM_MX4_MAX_TOKENS 64
#define QMM_MX4_MAX_TOP_K 32
#define QMM_MX4_MAX_EXPERTS 1024

/*
 * qmm_mx4_quantize: x (M, K) of x_dtype (QMM_F32, QMM_F16, QMM_BF16) to codes
 * (M, 16 B) and scales (M, B).  Every step is exact but the one rounding of each
 * code.  Signs are kept, of zeros too; a block of zeros has scale byte 0.  A
 * block that holds an infinity or a NaN has scale byte 255 and codes 0: it
 * stands for NaNs.
 * ldc is a multiple of 16 and codes start on 16 bytes.  The bytes of a row of
 * scales from B up to the next multiple of 4 or to lds, whichever is less, are
 * its padding: they are set to 0, the last row's too (lds = B has none).
 */
QMM_API qmm_status qmm_mx4_quantize(const void* x, int x_dtype, int64_t ldx, uint8_t* codes,
                                    int64_t ldc, uint8_t* scales, int64_t lds, int M, int K,
                                    void* stream);

/* qmm_mx4_dequantize: the values y (M, K) of y_dtype that codes and scales stand
 * for: exact, then rounded once to y's type.  Any alignment, any ld. */
QMM_API qmm_status qmm_mx4_dequantize(const uint8_t* codes, int64_t ldc, const uint8_t* scales,
                                      int64_t lds, void* y, int y_dtype, int64_t ldy, int M, int K,
                                      void* stream);

/* Bytes of a packed weight (N, K); 0 for invalid sizes. */
QMM_API size_t qmm_mx4_packed_bytes(int N, int K);

/*
 * qmm_mx4_pack: `batch` weights (N, K), codes (batch N, 16 B) and scales (batch N,
 * B) as above (any alignment and ld), to `batch` packed weights one after the other (offline).
 * W starts on 16 bytes.  A packed weight is the matrix cores' operand:
 *   columns (rows n of the weight) in strips of 16, K in chunks of 512 values (16
 *   blocks); a chunk of a strip is 4352 bytes, a strip's chunks follow each other.
 *   Codes: its bytes 1024 j + 16 L .. + 15, j < 4, L < 64, hold block 4 (L / 16) + j of
 *   column 16 strip + L % 16.
 *   Scales: its byte 4096 + 4 L + j is that block's scale.
 *   Blocks and columns that do not exist have codes 0 and scale byte 127.
 */
QMM_API qmm_status qmm_mx4_pack(const uint8_t* codes, int64_t ldc, const uint8_t* scales,
                                int64_t lds, void* W, int batch, int N, int K, void* stream);

/* Scratch of qmm_mx4_gemm: x laid out as the weight is.  Device memory, 16-byte aligned,
 * any contents; in use until the call's work on the stream is done.  0 for a few
 * values (which are quantized within the product's launch) and for invalid arguments. */
QMM_API size_t qmm_mx4_workspace_bytes(int M, int K, int x_dtype);

/*
 * qmm_mx4_gemm: y (M, N) of y_dtype (QMM_F32, QMM_F16, QMM_BF16) = x^ W^t.
 * x is either codes (x_dtype QMM_MX4, (M, 16 B), any alignment and ld) with their scales
 * sx (M, B), or values (sx NULL), which the call quantizes as qmm_mx4_quantize does.
 * W is a packed weight (N, K).  Sums are fp32, rounded to y's type once.
 */
QMM_API qmm_status qmm_mx4_gemm(const void* x, int x_dtype, int64_t ldx, const uint8_t* sx,
                                int64_t ldsx, const void* W, void* y, int y_dtype, int64_t ldy,
                                int M, int N, int K, void* workspace, size_t workspace_bytes,
                                void* stream);

/* Scratch of qmm_mx4_moe.  Device memory, 256-byte aligned, any contents; in use
 * until the call's work on the stream is done.  0 for invalid arguments. */
QMM_API size_t qmm_mx4_moe_workspace_bytes(int T, int D, int I, int E, int top_k, int x_dtype,
                                           int y_dtype);

/*
 * qmm_mx4_moe: y (T, D) of y_dtype for T <= QMM_MX4_MAX_TOKENS tokens x (T, D)
 * of x_dtype (QMM_F32, QMM_F16, QMM_BF16).  Wg and Wu are E packed weights (I, D)
 * one after the other, Wd E packed weights (D, I).  The activations are not
 * quantized: products are of x's own values and the weights', then of h's in fp32, whatever
 * y's type; sums are fp32.
 *   logits (T, E) of logits_dtype, not NULL: each token's top_k largest (the
 *     lower index of equal ones; NaN above everything), weighted by the softmax
 *     over them (renormalize 1) or over all (0).  A logit of minus infinity is
 *     never chosen; one that is NaN or plus infinity makes its token's y NaN.
 *   else ids (T, top_k) of ids_size bytes each (4 or 8) and weights (T, top_k) of
 *     weights_dtype, contiguous.  An index outside [0, E) counts for nothing;
 *     one that a token has twice counts with both weights.
 * A token without experts has y = 0.  T top_k D and T top_k I stay below
 * 2^28 - 2^16.
 */
QMM_API qmm_status qmm_mx4_moe(const void* x, int x_dtype, int64_t ldx, const void* Wg,
                               const void* Wu, const void* Wd, void* y, int y_dtype, int64_t ldy,
                               int T, int D, int I, int E, int top_k, int act, const void* logits,
                               int logits_dtype, int64_t ldl, int renormalize, const void* ids,
                               int ids_size, const void* weights, int weights_dtype,
                               void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* QMM_MX4_H */
