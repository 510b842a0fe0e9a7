// w8a8_api.cpp -- C ABI of the int8 x int8 operators (include/qmm_int8.h):
// argument checks before any HIP call, empty sums, dispatch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qmm_int8.h"
#include "w8a8_internal.h"

namespace {

using qmm::set_error;

#define QMM_REFUSE(status, ...) return static_cast<qmm_status>(set_error(status, __VA_ARGS__))

qmm_status done() { return static_cast<qmm_status>(qmm::clear_error()); }

qmm_status device_status(const char* fn, hipError_t e) {
  if (e != hipSuccess)
    QMM_REFUSE(QMM_ERR_DEVICE, "%s: HIP error %d (%s)", fn, (int)e, hipGetErrorString(e));
  return done();
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

constexpr int64_t kMaxLd = int64_t(1) << 22;  // 256 rows stay within 32-bit byte offsets
constexpr int kMaxK = 1 << 17;                // sums of code products fit 32 bits
constexpr int kMaxRows = INT32_MAX - 1024;    // indices within the last tile stay ints

int type_size(int t) { return t == QMM_F32 ? 4 : 2; }

qmm_status check_sizes(const char* fn, int M, int N, int K) {
  if (M < 0 || N < 0 || K < 0)
    QMM_REFUSE(QMM_ERR_ARG, "%s: negative size M=%d N=%d K=%d", fn, M, N, K);
  if (K >= kMaxK)
    QMM_REFUSE(QMM_ERR_UNSUPPORTED, "%s: K=%d too large for exact 32-bit sums (K < %d)", fn, K, kMaxK);
  if (M > kMaxRows || N > kMaxRows)
    QMM_REFUSE(QMM_ERR_UNSUPPORTED, "%s: M=%d or N=%d too large (at most %d)", fn, M, N, kMaxRows);
  return QMM_OK;
}

// A matrix of elements of `size` bytes (1: int8 codes, which start on 16
// bytes with rows of whole 16 bytes).
qmm_status check_matrix(const char* fn, const char* name, const void* p, int64_t ld, int cols,
                        int size) {
  if (p == nullptr) QMM_REFUSE(QMM_ERR_ARG, "%s: NULL %s", fn, name);
  if (ld < (cols > 1 ? cols : 1))
    QMM_REFUSE(QMM_ERR_ARG, "%s: leading dimension of %s is %lld, its rows have %d elements", fn,
               name, (long long)ld, cols);
  if (ld >= kMaxLd)
    QMM_REFUSE(QMM_ERR_UNSUPPORTED, "%s: leading dimension of %s too large (%lld, < %lld)", fn,
               name, (long long)ld, (long long)kMaxLd);
  if (size == 1) {
    if (ld % 16 != 0)
      QMM_REFUSE(QMM_ERR_UNSUPPORTED,
                 "%s: leading dimension of %s must be a multiple of 16 (got %lld)", fn, name,
                 (long long)ld);
    if (!aligned(p, 16)) QMM_REFUSE(QMM_ERR_ARG, "%s: %s must be 16-byte aligned", fn, name);
  } else if (!aligned(p, (uintptr_t)size)) {
    QMM_REFUSE(QMM_ERR_ARG, "%s: %s must be aligned to its elements (%d bytes)", fn, name, size);
  }
  return QMM_OK;
}

qmm_status check_vector(const char* fn, const char* name, const float* p) {
  if (p == nullptr) QMM_REFUSE(QMM_ERR_ARG, "%s: NULL %s", fn, name);
  if (!aligned(p, 4)) QMM_REFUSE(QMM_ERR_ARG, "%s: %s must be 4-byte aligned", fn, name);
  return QMM_OK;
}

bool value_type(int t) { return t == QMM_F32 || t == QMM_F16 || t == QMM_BF16; }

qmm_status check_act(const char* fn, int act) {
  if (act != QMM_SILU && act != QMM_GELU && act != QMM_GELU_TANH)
    QMM_REFUSE(QMM_ERR_ARG, "%s: act must be QMM_SILU, QMM_GELU or QMM_GELU_TANH (got %d)", fn, act);
  return QMM_OK;
}

qmm_status check_workspace(const char* fn, size_t need, const void* ws, size_t bytes,
                           uintptr_t align) {
  if (need == 0) return QMM_OK;
  if (ws == nullptr || bytes < need)
    QMM_REFUSE(QMM_ERR_ARG, "%s: workspace of %zu bytes needed (got %zu%s)", fn, need, bytes,
               ws ? "" : ", NULL");
  if (!aligned(ws, align))
    QMM_REFUSE(QMM_ERR_ARG, "%s: workspace must be %d-byte aligned", fn, (int)align);
  return QMM_OK;
}

#define QMM_CHECK(call)                  \
  do {                                   \
    const qmm_status st_ = (call);       \
    if (st_ != QMM_OK) return st_;       \
  } while (0)

int64_t code_ld(int K) { return qmm::round_up(K > 0 ? K : 1, 16); }

qmm_status forward(const char* fn, bool gated, const void* x, int x_dtype, int64_t ldx,
                   const float* sx, const int8_t* const (&w)[2], const float* const (&sw)[2],
                   int64_t ldw, void* y, int y_dtype, int64_t ldy, int M, int N, int K, int act,
                   void* ws, size_t ws_bytes, void* stream) {
  if (x_dtype != QMM_I8 && !value_type(x_dtype))
    QMM_REFUSE(QMM_ERR_ARG, "%s: x_dtype must be QMM_I8, QMM_F32, QMM_F16 or QMM_BF16 (got %d)", fn,
               x_dtype);
  if (!value_type(y_dtype))
    QMM_REFUSE(QMM_ERR_ARG, "%s: output type must be QMM_F32, QMM_F16 or QMM_BF16 (got %d)", fn, y_dtype);
  if (gated) QMM_CHECK(check_act(fn, act));
  QMM_CHECK(check_sizes(fn, M, N, K));
  if (x_dtype != QMM_I8 && sx != nullptr)
    QMM_REFUSE(QMM_ERR_ARG, "%s: sx goes with codes (x_dtype QMM_I8); it must be NULL for values", fn);
  if (M == 0 || N == 0) return done();
  const char* out = gated ? "h" : "y";
  QMM_CHECK(check_matrix(fn, out, y, ldy, N, type_size(y_dtype)));
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (K == 0)
    return device_status(fn, qmm::launch_fill_zero(y, type_size(y_dtype), ldy, M, N, s));
  QMM_CHECK(check_matrix(fn, "x", x, ldx, K, x_dtype == QMM_I8 ? 1 : type_size(x_dtype)));
  QMM_CHECK(check_matrix(fn, gated ? "Wg" : "W", w[0], ldw, K, 1));
  QMM_CHECK(check_vector(fn, gated ? "sg" : "sw", sw[0]));
  if (gated) {
    QMM_CHECK(check_matrix(fn, "Wu", w[1], ldw, K, 1));
    QMM_CHECK(check_vector(fn, "su", sw[1]));
  }
  qmm::W8A8Args a{};
  a.w[0] = w[0], a.w[1] = w[1];
  a.sw[0] = sw[0], a.sw[1] = sw[1];
  a.ldw = ldw;
  a.y = y, a.y_dtype = y_dtype, a.ldy = ldy;
  a.M = M, a.N = N, a.K = K;
  a.gated = gated, a.act = act;
  a.stream = s;
  if (x_dtype == QMM_I8) QMM_CHECK(check_vector(fn, "sx", sx));
  else QMM_CHECK(check_workspace(fn, qmm_w8a8_workspace_bytes(M, K, x_dtype), ws, ws_bytes, 16));
  if (qmm::rows_fits(M, K)) {
    a.sx = sx;
    return device_status(fn, qmm::launch_rows(a, x, x_dtype, ldx));
  }
  if (x_dtype == QMM_I8) {
    a.x = static_cast<const int8_t*>(x);
    a.ldx = ldx;
    a.sx = sx;
  } else {
    int8_t* xq = static_cast<int8_t*>(ws);
    a.ldx = code_ld(K);
    float* scale = reinterpret_cast<float*>(xq + (size_t)M * a.ldx);
    const hipError_t e = qmm::launch_quantize_tokens(x, x_dtype, ldx, xq, a.ldx, scale, M, K, s);
    if (e != hipSuccess) return device_status(fn, e);
    a.x = xq;
    a.sx = scale;
  }
  return device_status(fn, qmm::launch_w8a8(a));
}

// the contracted axes become leading dimensions of 16-bit operands
bool backward_fits(int M, int N, bool gated) {
  return (int64_t)N * (gated ? 2 : 1) < kMaxLd / 2 - 256 && M < kMaxLd / 2 - 256;
}

qmm_status backward(const char* fn, bool gated, const void* dy, int dtype, int64_t lddy,
                    const int8_t* x, int64_t ldx, const float* sx, const int8_t* const (&w)[2],
                    const float* const (&sw)[2], int64_t ldw, void* dx, int64_t lddx,
                    void* const (&dw)[2], int64_t lddw, int M, int N, int K, int act, void* ws,
                    size_t ws_bytes, void* stream) {
  if (dtype != QMM_F16 && dtype != QMM_BF16)
    QMM_REFUSE(QMM_ERR_ARG, "%s: dtype must be QMM_F16 or QMM_BF16 (got %d)", fn, dtype);
  if (gated) QMM_CHECK(check_act(fn, act));
  QMM_CHECK(check_sizes(fn, M, N, K));
  if (!backward_fits(M, N, gated))
    QMM_REFUSE(QMM_ERR_UNSUPPORTED, "%s: M=%d or N=%d too large", fn, M, N);
  const bool wgrad = dw[0] != nullptr;
  if (gated && (dw[1] != nullptr) != wgrad)
    QMM_REFUSE(QMM_ERR_ARG, "%s: dWg and dWu are given together or not at all", fn);
  if (K == 0 || (M == 0 && (N == 0 || !wgrad))) return done();
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int parts = gated ? 2 : 1;
  if (M > 0) QMM_CHECK(check_matrix(fn, "dx", dx, lddx, K, 2));
  if (wgrad && N > 0) {
    QMM_CHECK(check_matrix(fn, gated ? "dWg" : "dW", dw[0], lddw, K, 2));
    if (gated) QMM_CHECK(check_matrix(fn, "dWu", dw[1], lddw, K, 2));
  }
  if (N == 0) return device_status(fn, qmm::launch_fill_zero(dx, 2, lddx, M, K, s));
  if (M == 0) {
    hipError_t e = hipSuccess;
    for (int i = 0; i < parts && e == hipSuccess; ++i)
      e = qmm::launch_fill_zero(dw[i], 2, lddw, N, K, s);
    return device_status(fn, e);
  }
  QMM_CHECK(check_matrix(fn, gated ? "dh" : "dy", dy, lddy, N, 2));
  QMM_CHECK(check_matrix(fn, gated ? "Wg" : "W", w[0], ldw, K, 1));
  QMM_CHECK(check_vector(fn, gated ? "sg" : "sw", sw[0]));
  if (gated) {
    QMM_CHECK(check_matrix(fn, "Wu", w[1], ldw, K, 1));
    QMM_CHECK(check_vector(fn, "su", sw[1]));
  }
  if (gated || wgrad) {
    QMM_CHECK(check_matrix(fn, "xq", x, ldx, K, 1));
    QMM_CHECK(check_vector(fn, "sx", sx));
  }
  const qmm::BackwardPlan p = qmm::plan_backward(M, N, K, gated, wgrad);
  QMM_CHECK(check_workspace(fn, p.bytes, ws, ws_bytes, 256));
  qmm::BackwardArgs a{};
  a.dy = dy, a.dtype = dtype, a.lddy = lddy;
  a.x = x, a.ldx = ldx, a.sx = sx;
  a.w[0] = w[0], a.w[1] = w[1];
  a.sw[0] = sw[0], a.sw[1] = sw[1];
  a.ldw = ldw;
  a.dx = dx, a.lddx = lddx;
  a.dw[0] = dw[0], a.dw[1] = dw[1], a.lddw = lddw;
  a.M = M, a.N = N, a.K = K;
  a.gated = gated, a.act = act;
  a.ws = ws;
  a.stream = s;
  return device_status(fn, qmm::launch_backward(a, p));
}

}  // namespace

namespace qmm {

hipError_t launch_w8a8(const W8A8Args& a) {
  TileArgs t{};
  t.a = a.x;
  t.lda = a.ldx;
  t.b[0] = a.w[0], t.b[1] = a.w[1];
  t.ldb = a.ldw;
  t.M = a.M, t.N = a.N, t.kb = a.K;
  t.sa = a.sx;
  t.sb[0] = a.sw[0], t.sb[1] = a.sw[1];
  t.y = a.y, t.y_dtype = a.y_dtype, t.ldy = a.ldy;
  t.act = a.act;
  if (skinny_fits(a.M)) return launch_skinny(t, a.gated, a.stream);
  hipError_t e = hipSuccess;
  for (int64_t m = 0; m < a.M && e == hipSuccess; m += kMaxLaunchRows) {
    t.a = a.x + m * a.ldx;
    t.sa = a.sx + m;
    t.y = static_cast<char*>(a.y) + m * a.ldy * type_size(a.y_dtype);
    t.M = (int)(a.M - m < kMaxLaunchRows ? a.M - m : kMaxLaunchRows);
    e = a.gated ? launch_tile_gated(t, a.stream) : launch_tile_scale(t, a.stream);
  }
  return e;
}

}  // namespace qmm

extern "C" {

qmm_status qmm_quantize_tokens(const void* x, int x_dtype, int64_t ldx, int8_t* xq, int64_t ldxq,
                               float* sx, int M, int K, void* stream) {
  const char* fn = "qmm_quantize_tokens";
  if (!value_type(x_dtype))
    QMM_REFUSE(QMM_ERR_ARG, "%s: x_dtype must be QMM_F32, QMM_F16 or QMM_BF16 (got %d)", fn, x_dtype);
  QMM_CHECK(check_sizes(fn, M, 0, K));
  if (M == 0) return done();
  QMM_CHECK(check_vector(fn, "sx", sx));
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (K == 0) return device_status(fn, qmm::launch_fill_zero(sx, 4, 1, M, 1, s));
  QMM_CHECK(check_matrix(fn, "x", x, ldx, K, type_size(x_dtype)));
  QMM_CHECK(check_matrix(fn, "xq", xq, ldxq, K, 1));
  return device_status(fn, qmm::launch_quantize_tokens(x, x_dtype, ldx, xq, ldxq, sx, M, K, s));
}

size_t qmm_w8a8_workspace_bytes(int M, int K, int x_dtype) {
  if (M <= 0 || M > kMaxRows || K <= 0 || K >= kMaxK || !value_type(x_dtype)) return 0;
  if (qmm::rows_fits(M, K)) return 0;  // quantized in LDS
  return (size_t)M * code_ld(K) + (size_t)M * 4;
}

qmm_status qmm_w8a8_gemm(const void* x, int x_dtype, int64_t ldx, const float* sx, const int8_t* W,
                         int64_t ldw, const float* sw, void* y, int y_dtype, int64_t ldy, int M,
                         int N, int K, void* workspace, size_t workspace_bytes, void* stream) {
  return forward("qmm_w8a8_gemm", false, x, x_dtype, ldx, sx, {W, nullptr}, {sw, nullptr}, ldw, y,
                 y_dtype, ldy, M, N, K, 0, workspace, workspace_bytes, stream);
}

qmm_status qmm_w8a8_gated(const void* x, int x_dtype, int64_t ldx, const float* sx,
                          const int8_t* Wg, const float* sg, const int8_t* Wu, const float* su,
                          int64_t ldw, void* h, int h_dtype, int64_t ldh, int M, int N, int K,
                          int act, void* workspace, size_t workspace_bytes, void* stream) {
  return forward("qmm_w8a8_gated", true, x, x_dtype, ldx, sx, {Wg, Wu}, {sg, su}, ldw, h, h_dtype,
                 ldh, M, N, K, act, workspace, workspace_bytes, stream);
}

size_t qmm_w8a8_backward_workspace_bytes(int M, int N, int K, int gated, int weight_grad) {
  if (M <= 0 || N <= 0 || K <= 0 || K >= kMaxK || !backward_fits(M, N, gated != 0)) return 0;
  return qmm::plan_backward(M, N, K, gated != 0, weight_grad != 0).bytes;
}

qmm_status qmm_w8a8_gemm_backward(const void* dy, int dtype, int64_t lddy, const int8_t* xq,
                                  int64_t ldx, const float* sx, const int8_t* W, int64_t ldw,
                                  const float* sw, void* dx, int64_t lddx, void* dW, int64_t lddw,
                                  int M, int N, int K, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  return backward("qmm_w8a8_gemm_backward", false, dy, dtype, lddy, xq, ldx, sx, {W, nullptr},
                  {sw, nullptr}, ldw, dx, lddx, {dW, nullptr}, lddw, M, N, K, 0, workspace,
                  workspace_bytes, stream);
}

qmm_status qmm_w8a8_gated_backward(const void* dh, int dtype, int64_t lddh, const int8_t* xq,
                                   int64_t ldx, const float* sx, const int8_t* Wg, const float* sg,
                                   const int8_t* Wu, const float* su, int64_t ldw, void* dx,
                                   int64_t lddx, void* dWg, void* dWu, int64_t lddw, int M, int N,
                                   int K, int act, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  return backward("qmm_w8a8_gated_backward", true, dh, dtype, lddh, xq, ldx, sx, {Wg, Wu}, {sg, su},
                  ldw, dx, lddx, {dWg, dWu}, lddw, M, N, K, act, workspace, workspace_bytes, stream);
}

}  // extern "C"
