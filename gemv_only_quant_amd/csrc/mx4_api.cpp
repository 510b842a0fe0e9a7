// mx4_api.cpp -- C ABI of the microscaled 4-bit operators (include/qmm_mx4.h):
// argument checks before any HIP call, empty sums, dispatch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qmm_mx4.h"
#include "mx4_internal.h"

namespace {

using qmm::set_error;

#define QMM_REFUSE(status, ...) return static_cast<qmm_status>(set_error(status, __VA_ARGS__))
#define QMM_CHECK(call)                  \
  do {                                   \
    const qmm_status st_ = (call);       \
    if (st_ != QMM_OK) return st_;       \
  } while (0)

qmm_status done() { return static_cast<qmm_status>(qmm::clear_error()); }

qmm_status device_status(const char* fn, hipError_t e) {
  if (e != hipSuccess)
    QMM_REFUSE(QMM_ERR_DEVICE, "%s: HIP error %d (%s)", fn, (int)e, hipGetErrorString(e));
  return done();
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool value_type(int t) { return t == QMM_F32 || t == QMM_F16 || t == QMM_BF16; }
int type_size(int t) { return t == QMM_F32 ? 4 : 2; }

constexpr int64_t kMaxLd = int64_t(1) << 22;  // 256 rows stay within 32-bit byte offsets
constexpr int kMaxK = 1 << 20;                // a packed strip's bytes fit 32 bits
constexpr int kMaxRows = INT32_MAX - 1024;    // indices within the last tile stay ints

qmm_status check_type(const char* fn, const char* name, int t) {
  if (!value_type(t))
    QMM_REFUSE(QMM_ERR_ARG, "%s: %s must be QMM_F32, QMM_F16 or QMM_BF16 (got %d)", fn, name, t);
  return QMM_OK;
}

qmm_status check_sizes(const char* fn, int M, int N, int K) {
  if (M < 0 || N < 0 || K < 0)
    QMM_REFUSE(QMM_ERR_ARG, "%s: negative size M=%d N=%d K=%d", fn, M, N, K);
  if (K >= kMaxK) QMM_REFUSE(QMM_ERR_UNSUPPORTED, "%s: K=%d too large (K < %d)", fn, K, kMaxK);
  if (M > kMaxRows || N > kMaxRows)
    QMM_REFUSE(QMM_ERR_UNSUPPORTED, "%s: M=%d or N=%d too large (at most %d)", fn, M, N, kMaxRows);
  return QMM_OK;
}

// A matrix whose rows have `cols` elements of `size` bytes, aligned to `align` bytes, its
// leading dimension a multiple of `whole`.
qmm_status check_matrix(const char* fn, const char* name, const void* p, int64_t ld, int64_t cols,
                        int align, int whole) {
  if (p == nullptr) QMM_REFUSE(QMM_ERR_ARG, "%s: NULL %s", fn, name);
  if (ld < (cols > 1 ? cols : 1))
    QMM_REFUSE(QMM_ERR_ARG, "%s: leading dimension of %s is %lld, its rows have %lld elements", fn,
               name, (long long)ld, (long long)cols);
  if (ld >= kMaxLd)
    QMM_REFUSE(QMM_ERR_UNSUPPORTED, "%s: leading dimension of %s too large (%lld, < %lld)", fn,
               name, (long long)ld, (long long)kMaxLd);
  if (ld % whole != 0)
    QMM_REFUSE(QMM_ERR_UNSUPPORTED, "%s: leading dimension of %s must be a multiple of %d (got %lld)",
               fn, name, whole, (long long)ld);
  if (!aligned(p, (uintptr_t)align))
    QMM_REFUSE(QMM_ERR_ARG, "%s: %s must be %d-byte aligned", fn, name, align);
  return QMM_OK;
}

qmm_status check_values(const char* fn, const char* name, const void* p, int64_t ld, int cols, int t) {
  return check_matrix(fn, name, p, ld, cols, type_size(t), 1);
}

qmm_status check_packed(const char* fn, const char* name, const void* p) {
  if (p == nullptr) QMM_REFUSE(QMM_ERR_ARG, "%s: NULL %s", fn, name);
  if (!aligned(p, 16)) QMM_REFUSE(QMM_ERR_ARG, "%s: %s must be 16-byte aligned", fn, name);
  return QMM_OK;
}

qmm_status check_workspace(const char* fn, size_t need, const void* ws, size_t bytes, uintptr_t align) {
  if (need == 0) return QMM_OK;
  if (ws == nullptr || bytes < need)
    QMM_REFUSE(QMM_ERR_ARG, "%s: workspace of %zu bytes needed (got %zu%s)", fn, need, bytes,
               ws ? "" : ", NULL");
  if (!aligned(ws, align))
    QMM_REFUSE(QMM_ERR_ARG, "%s: workspace must be %d-byte aligned", fn, (int)align);
  return QMM_OK;
}

constexpr int64_t kMaxHidden = (int64_t(1) << 28) - (int64_t(1) << 16);  // a part of h, and z, fit 32-bit byte offsets

bool moe_sizes_ok(int T, int D, int I, int E, int top_k) {
  return T >= 0 && D >= 0 && I >= 0 && E >= 0 && top_k >= 0 && T <= QMM_MX4_MAX_TOKENS && D < kMaxK &&
         I < kMaxK && E <= QMM_MX4_MAX_EXPERTS && top_k <= QMM_MX4_MAX_TOP_K &&
         (int64_t)T * top_k * (I > D ? I : D) < kMaxHidden;
}

}  // namespace

extern "C" {

qmm_status qmm_mx4_quantize(const void* x, int x_dtype, int64_t ldx, uint8_t* codes, int64_t ldc,
                            uint8_t* scales, int64_t lds, int M, int K, void* stream) {
  const char* fn = "qmm_mx4_quantize";
  QMM_CHECK(check_type(fn, "x_dtype", x_dtype));
  QMM_CHECK(check_sizes(fn, M, 0, K));
  if (M == 0 || K == 0) return done();
  const int B = qmm::mx4_blocks(K);
  QMM_CHECK(check_values(fn, "x", x, ldx, K, x_dtype));
  QMM_CHECK(check_matrix(fn, "codes", codes, ldc, 16 * (int64_t)B, 16, 16));
  QMM_CHECK(check_matrix(fn, "scales", scales, lds, B, 1, 1));
  return device_status(fn, qmm::launch_mx4_quantize(x, x_dtype, ldx, codes, ldc, scales, lds, M, K,
                                                    reinterpret_cast<hipStream_t>(stream)));
}

qmm_status qmm_mx4_dequantize(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds,
                              void* y, int y_dtype, int64_t ldy, int M, int K, void* stream) {
  const char* fn = "qmm_mx4_dequantize";
  QMM_CHECK(check_type(fn, "y_dtype", y_dtype));
  QMM_CHECK(check_sizes(fn, M, 0, K));
  if (M == 0 || K == 0) return done();
  const int B = qmm::mx4_blocks(K);
  QMM_CHECK(check_matrix(fn, "codes", codes, ldc, 16 * (int64_t)B, 1, 1));
  QMM_CHECK(check_matrix(fn, "scales", scales, lds, B, 1, 1));
  QMM_CHECK(check_values(fn, "y", y, ldy, K, y_dtype));
  return device_status(fn, qmm::launch_mx4_dequantize(codes, ldc, scales, lds, y, y_dtype, ldy, M, K,
                                                      reinterpret_cast<hipStream_t>(stream)));
}

size_t qmm_mx4_packed_bytes(int N, int K) {
  if (N <= 0 || K <= 0 || N > kMaxRows || K >= kMaxK) return 0;
  return (size_t)qmm::mx4_weight_bytes(N, K);
}

qmm_status qmm_mx4_pack(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, void* W,
                        int batch, int N, int K, void* stream) {
  const char* fn = "qmm_mx4_pack";
  if (batch < 0) QMM_REFUSE(QMM_ERR_ARG, "%s: negative batch %d", fn, batch);
  QMM_CHECK(check_sizes(fn, 0, N, K));
  if ((int64_t)batch * ((N + 15) / 16) > kMaxRows)
    QMM_REFUSE(QMM_ERR_UNSUPPORTED, "%s: batch=%d of N=%d too large", fn, batch, N);
  if (batch == 0 || N == 0 || K == 0) return done();
  const int B = qmm::mx4_blocks(K);
  QMM_CHECK(check_matrix(fn, "codes", codes, ldc, 16 * (int64_t)B, 1, 1));
  QMM_CHECK(check_matrix(fn, "scales", scales, lds, B, 1, 1));
  QMM_CHECK(check_packed(fn, "W", W));
  return device_status(fn, qmm::launch_mx4_pack(codes, ldc, scales, lds, W, batch, N, K,
                                                reinterpret_cast<hipStream_t>(stream)));
}

size_t qmm_mx4_workspace_bytes(int M, int K, int x_dtype) {
  if (M <= 0 || M > kMaxRows || K <= 0 || K >= kMaxK) return 0;
  if (x_dtype != QMM_MX4 && !value_type(x_dtype)) return 0;
  if (x_dtype != QMM_MX4 && qmm::mx4_rows_fits(M, K)) return 0;  // quantized in LDS
  return (size_t)qmm::mx4_weight_bytes(M, K);
}

qmm_status qmm_mx4_gemm(const void* x, int x_dtype, int64_t ldx, const uint8_t* sx, int64_t ldsx,
                        const void* W, void* y, int y_dtype, int64_t ldy, int M, int N, int K,
                        void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "qmm_mx4_gemm";
  const bool coded = x_dtype == QMM_MX4;
  if (!coded && !value_type(x_dtype))
    QMM_REFUSE(QMM_ERR_ARG, "%s: x_dtype must be QMM_MX4, QMM_F32, QMM_F16 or QMM_BF16 (got %d)", fn,
               x_dtype);
  QMM_CHECK(check_type(fn, "y_dtype", y_dtype));
  QMM_CHECK(check_sizes(fn, M, N, K));
  if (!coded && sx != nullptr)
    QMM_REFUSE(QMM_ERR_ARG, "%s: sx goes with codes (x_dtype QMM_MX4); it must be NULL for values", fn);
  if (M == 0 || N == 0) return done();
  QMM_CHECK(check_values(fn, "y", y, ldy, N, y_dtype));
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (K == 0) return device_status(fn, qmm::launch_fill_zero(y, type_size(y_dtype), ldy, M, N, s));
  const int B = qmm::mx4_blocks(K);
  if (coded) {
    QMM_CHECK(check_matrix(fn, "x", x, ldx, 16 * (int64_t)B, 1, 1));
    QMM_CHECK(check_matrix(fn, "sx", sx, ldsx, B, 1, 1));
  } else {
    QMM_CHECK(check_values(fn, "x", x, ldx, K, x_dtype));
  }
  QMM_CHECK(check_packed(fn, "W", W));
  QMM_CHECK(check_workspace(fn, qmm_mx4_workspace_bytes(M, K, x_dtype), workspace, workspace_bytes, 16));
  qmm::Mx4Args a{};
  a.w = static_cast<const uint8_t*>(W);
  a.y = y, a.y_dtype = y_dtype, a.ldy = ldy;
  a.M = M, a.N = N, a.K = K;
  if (!coded && qmm::mx4_rows_fits(M, K)) return device_status(fn, qmm::launch_mx4_rows(a, x, x_dtype, ldx, s));
  // x in the matrix cores' layout, as the weight
  uint8_t* packed = static_cast<uint8_t*>(workspace);
  a.a = packed;
  hipError_t e = coded ? qmm::launch_mx4_pack(static_cast<const uint8_t*>(x), ldx, sx, ldsx, packed, 1, M, K, s)
                       : qmm::launch_mx4_quantize_packed(x, x_dtype, ldx, packed, M, K, s);
  if (e == hipSuccess) e = qmm::mx4_skinny_fits(M, N) ? qmm::launch_mx4_skinny(a, s) : qmm::launch_mx4_large(a, s);
  return device_status(fn, e);
}

size_t qmm_mx4_moe_workspace_bytes(int T, int D, int I, int E, int top_k, int x_dtype, int y_dtype) {
  if (!moe_sizes_ok(T, D, I, E, top_k) || !value_type(x_dtype) || !value_type(y_dtype)) return 0;
  if (T == 0 || D == 0 || I == 0 || E == 0 || top_k == 0) return 0;
  return qmm::plan_moe(T, D, I, E, top_k, x_dtype).bytes;
}

qmm_status qmm_mx4_moe(const void* x, int x_dtype, int64_t ldx, const void* Wg, const void* Wu,
                       const void* Wd, void* y, int y_dtype, int64_t ldy, int T, int D, int I, int E,
                       int top_k, int act, const void* logits, int logits_dtype, int64_t ldl,
                       int renormalize, const void* ids, int ids_size, const void* weights,
                       int weights_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "qmm_mx4_moe";
  QMM_CHECK(check_type(fn, "x_dtype", x_dtype));
  QMM_CHECK(check_type(fn, "y_dtype", y_dtype));
  if (act != QMM_SILU && act != QMM_GELU && act != QMM_GELU_TANH)
    QMM_REFUSE(QMM_ERR_ARG, "%s: act must be QMM_SILU, QMM_GELU or QMM_GELU_TANH (got %d)", fn, act);
  if (T < 0 || D < 0 || I < 0 || E < 0 || top_k < 0)
    QMM_REFUSE(QMM_ERR_ARG, "%s: negative size T=%d D=%d I=%d E=%d top_k=%d", fn, T, D, I, E, top_k);
  if (!moe_sizes_ok(T, D, I, E, top_k))
    QMM_REFUSE(QMM_ERR_UNSUPPORTED,
               "%s: T=%d (at most %d), E=%d (%d), top_k=%d (%d), D=%d or I=%d (< %d) or T top_k max(D, I) (< %lld) too large",
               fn, T, QMM_MX4_MAX_TOKENS, E, QMM_MX4_MAX_EXPERTS, top_k, QMM_MX4_MAX_TOP_K, D, I, kMaxK,
               (long long)kMaxHidden);
  if (logits != nullptr) {
    QMM_CHECK(check_type(fn, "logits_dtype", logits_dtype));
    if (ids != nullptr || weights != nullptr)
      QMM_REFUSE(QMM_ERR_ARG, "%s: logits, or ids and weights, not both", fn);
    if (top_k > E) QMM_REFUSE(QMM_ERR_ARG, "%s: top_k=%d of E=%d experts", fn, top_k, E);
    if (renormalize != 0 && renormalize != 1)
      QMM_REFUSE(QMM_ERR_ARG, "%s: renormalize must be 0 or 1 (got %d)", fn, renormalize);
  } else if (ids != nullptr || weights != nullptr) {
    QMM_CHECK(check_type(fn, "weights_dtype", weights_dtype));
    if (ids_size != 4 && ids_size != 8)
      QMM_REFUSE(QMM_ERR_ARG, "%s: ids_size must be 4 or 8 (got %d)", fn, ids_size);
  }
  if (T == 0 || D == 0) return done();
  QMM_CHECK(check_values(fn, "y", y, ldy, D, y_dtype));
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (I == 0 || E == 0 || top_k == 0)
    return device_status(fn, qmm::launch_fill_zero(y, type_size(y_dtype), ldy, T, D, s));
  QMM_CHECK(check_values(fn, "x", x, ldx, D, x_dtype));
  QMM_CHECK(check_packed(fn, "Wg", Wg));
  QMM_CHECK(check_packed(fn, "Wu", Wu));
  QMM_CHECK(check_packed(fn, "Wd", Wd));
  if (logits != nullptr) {
    QMM_CHECK(check_values(fn, "logits", logits, ldl, E, logits_dtype));
  } else {
    if (ids == nullptr || weights == nullptr)
      QMM_REFUSE(QMM_ERR_ARG, "%s: logits, or ids and weights, must be given", fn);
    if (!aligned(ids, (uintptr_t)ids_size) || !aligned(weights, (uintptr_t)type_size(weights_dtype)))
      QMM_REFUSE(QMM_ERR_ARG, "%s: ids and weights must be aligned to their elements", fn);
  }
  const qmm::MoePlan p = qmm::plan_moe(T, D, I, E, top_k, x_dtype);
  QMM_CHECK(check_workspace(fn, p.bytes, workspace, workspace_bytes, 256));
  qmm::MoeArgs a{};
  a.x = x, a.x_dtype = x_dtype, a.ldx = ldx;
  a.wg = static_cast<const uint8_t*>(Wg);
  a.wu = static_cast<const uint8_t*>(Wu);
  a.wd = static_cast<const uint8_t*>(Wd);
  a.y = y, a.y_dtype = y_dtype, a.ldy = ldy;
  a.T = T, a.D = D, a.I = I, a.E = E, a.top_k = top_k, a.act = act;
  a.logits = logits, a.logits_dtype = logits_dtype, a.ldl = ldl, a.renormalize = renormalize;
  a.ids = ids, a.ids_size = ids_size, a.weights = weights, a.weights_dtype = weights_dtype;
  a.ws = workspace;
  return device_status(fn, qmm::launch_mx4_moe(a, p, s));
}

}  // extern "C"
