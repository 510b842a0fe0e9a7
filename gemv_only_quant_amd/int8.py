"""Python binding of the int8 x int8 operators (include/qmm_int8.h): the
per-token quantizer, the product with scales for each token and channel, the
gated feed-forward block on it, and their gradients.

    xq, sx = quantize_tokens(x)                       # (M, K) -> int8 codes, (M,) scales
    y = w8a8_gemm(x, W, sw)                           # x values, quantized by the call
    y = w8a8_gemm(xq, W, sw, sx=sx)                   # or codes with their scales
    h = w8a8_gated(x, Wg, sg, Wu, su, act="silu")     # act(x^ Wg^t) * (x^ Wu^t)
    dx, dW = w8a8_gemm_backward(dy, xq, sx, W, sw)
    dx, dWg, dWu = w8a8_gated_backward(dh, xq, sx, Wg, sg, Wu, su, act="silu")

Matrices are 2-D tensors with unit column stride (a slice of the columns of a
wider tensor will do); int8 ones have a row stride that is a multiple of 16
and start on 16 bytes.  All of a call's tensors sit on one GPU; the work goes
to that GPU's current stream and the scratch comes from torch's allocator on
that stream, so tensors in use on another stream need the usual wait_stream
or record_stream.  Nothing here is an autograd function: the backward calls
are what one's backward would call.  A call whose operands require gradients warns
that it passes none on, unless gradients are off.
"""
import ctypes
import warnings

import torch

from . import (QMM_BF16, QMM_ERR_ARG, QMM_ERR_UNSUPPORTED, QMM_F16, QMM_F32, QmmError, _check,
               _lib)

QMM_I8 = 3  # x_dtype of activations that are codes already
QMM_SILU, QMM_GELU, QMM_GELU_TANH = 0, 1, 2
ACTIVATIONS = {"silu": QMM_SILU, "gelu": QMM_GELU, "gelu_tanh": QMM_GELU_TANH}

_P, _I, _L, _S = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
_lib.qmm_quantize_tokens.argtypes = [_P, _I, _L, _P, _L, _P, _I, _I, _P]
_lib.qmm_w8a8_workspace_bytes.argtypes = [_I, _I, _I]
_lib.qmm_w8a8_workspace_bytes.restype = _S
_lib.qmm_w8a8_gemm.argtypes = [_P, _I, _L, _P, _P, _L, _P, _P, _I, _L, _I, _I, _I, _P, _S, _P]
_lib.qmm_w8a8_gated.argtypes = [_P, _I, _L, _P, _P, _P, _P, _P, _L, _P, _I, _L, _I, _I, _I, _I,
                                _P, _S, _P]
_lib.qmm_w8a8_backward_workspace_bytes.argtypes = [_I, _I, _I, _I, _I]
_lib.qmm_w8a8_backward_workspace_bytes.restype = _S
_lib.qmm_w8a8_gemm_backward.argtypes = [_P, _I, _L, _P, _L, _P, _P, _L, _P, _P, _L, _P, _L, _I,
                                        _I, _I, _P, _S, _P]
_lib.qmm_w8a8_gated_backward.argtypes = [_P, _I, _L, _P, _L, _P, _P, _P, _P, _P, _L, _P, _L, _P,
                                         _P, _L, _I, _I, _I, _I, _P, _S, _P]

EXPORTS_INT8 = ("qmm_quantize_tokens", "qmm_w8a8_workspace_bytes", "qmm_w8a8_gemm",
                "qmm_w8a8_gated", "qmm_w8a8_backward_workspace_bytes", "qmm_w8a8_gemm_backward",
                "qmm_w8a8_gated_backward")

_INT_MAX = (1 << 31) - 1
_CODES = {torch.float32: QMM_F32, torch.float16: QMM_F16, torch.bfloat16: QMM_BF16}


def _refuse(fn, text, status=QMM_ERR_ARG):
    raise QmmError(status, f"{fn}: {text}")


def _matrix(fn, name, t, shape=None):
    """(pointer, leading dimension) of a 2-D tensor with unit column stride."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        _refuse(fn, f"{name} must be a 2-D tensor")
    rows, cols = t.shape
    if rows > _INT_MAX or cols > _INT_MAX:  # ctypes would pass on the low 32 bits
        _refuse(fn, f"{name} is too large ({rows} x {cols})", QMM_ERR_UNSUPPORTED)
    if shape is not None and (rows, cols) != shape:
        _refuse(fn, f"{name} must be {tuple(shape)}, got {(rows, cols)}")
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        _refuse(fn, f"{name} must have unit column stride (got strides {t.stride()})")
    if rows <= 1:  # a single row's stride is never used
        ld = max(cols, 1)
    elif cols == 1 and ld < 1:
        _refuse(fn, f"{name} has rows that overlap (strides {t.stride()})")
    return t.data_ptr(), ld


def _int8_matrix(fn, name, t, shape=None):
    """As _matrix, for int8 codes: rows of whole 16 bytes, of which the last
    row's must be readable too."""
    if isinstance(t, torch.Tensor) and t.dtype != torch.int8:
        _refuse(fn, f"{name} must be int8, got {t.dtype}")
    ptr, ld = _matrix(fn, name, t, shape)
    rows, cols = t.shape
    if rows <= 1:
        ld = -(-ld // 16) * 16
    if cols % 16 and rows:
        end = t.storage_offset() + (rows - 1) * ld + -(-cols // 16) * 16
        if end > t.untyped_storage().nbytes():
            _refuse(fn, f"{name} has rows of {cols} codes: its storage must hold whole 16 bytes "
                        f"for each row (pad the rows; quantize_tokens does)", QMM_ERR_UNSUPPORTED)
    return ptr, ld


def _scale(fn, name, t, n):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32:
        _refuse(fn, f"{name} must be a float32 tensor")
    if t.numel() != n or not t.is_contiguous():
        _refuse(fn, f"{name} must hold {n} contiguous values (got {tuple(t.shape)})")
    return t.data_ptr()


def _one_gpu(fn, *tensors):
    """Index of the GPU that holds all of them; warns where gradients end here."""
    index = None
    for t in tensors:
        if t is None:
            continue
        i = t.get_device()
        if i != index:
            if not t.is_cuda:
                _refuse(fn, f"operands must be GPU tensors (got one on {t.device})")
            if index is not None:
                _refuse(fn, f"operands on different GPUs ({index} and {i})")
            index = i
        if t.requires_grad and torch.is_grad_enabled():
            warnings.warn(f"{fn}: an operand requires gradients, and this call passes none on; call it and its "
                          f"backward call from a torch.autograd.Function, or under torch.no_grad()", stacklevel=3)
    return index


def _run(index, call):
    """call(stream) with the GPU current, on its current stream."""
    if index == torch.cuda.current_device():
        _check(call(torch.cuda.current_stream(index).cuda_stream))
    else:
        with torch.cuda.device(index):
            _check(call(torch.cuda.current_stream(index).cuda_stream))


def _float_type(fn, name, dtype, types=_CODES):
    if dtype not in types:
        want = ", ".join(str(d).replace("torch.", "") for d in types)
        _refuse(fn, f"{name} must be one of {want}, got {dtype}")
    return types[dtype]


def _output(fn, name, out, out_dtype, shape, device):
    """(tensor, type code, pointer, leading dimension): `out` checked, or a new
    tensor."""
    if out is None:
        code = _float_type(fn, "out_dtype", out_dtype)
        out = torch.empty(shape, dtype=out_dtype, device=device)
        return out, code, out.data_ptr(), max(shape[1], 1)
    ptr, ld = _matrix(fn, name, out, shape)
    return out, _float_type(fn, name, out.dtype), ptr, ld


def _act(fn, act):
    if act not in ACTIVATIONS:
        _refuse(fn, f"act must be one of {', '.join(ACTIVATIONS)}, got {act!r}")
    return ACTIVATIONS[act]


def quantize_tokens(x):
    """x (M, K) float32 / float16 / bfloat16 -> (codes (M, K) int8, scales (M,)
    float32).  The codes are a view of rows padded to 16 bytes."""
    fn = "qmm_quantize_tokens"
    px, ldx = _matrix(fn, "x", x)
    code = _float_type(fn, "x", x.dtype)
    index = _one_gpu(fn, x)
    M, K = x.shape
    ld = max(16, -(-K // 16) * 16)
    q = torch.empty((M, ld), dtype=torch.int8, device=x.device)
    s = torch.empty((M,), dtype=torch.float32, device=x.device)
    _run(index, lambda st: _lib.qmm_quantize_tokens(px, code, ldx, q.data_ptr(), ld, s.data_ptr(),
                                                    M, K, st))
    return q[:, :K], s


def _left(fn, x, sx):
    """The left operand: (type code, pointer, leading dimension, scales'
    pointer, bytes of scratch) of codes with scales or of values."""
    if isinstance(x, torch.Tensor) and x.dtype == torch.int8:
        px, ldx = _int8_matrix(fn, "x", x)
        if sx is None:
            _refuse(fn, "int8 x needs its scales (sx)")
        return QMM_I8, px, ldx, _scale(fn, "sx", sx, x.shape[0]), 0
    px, ldx = _matrix(fn, "x", x)
    if sx is not None:
        _refuse(fn, "sx goes with int8 x")
    code = _float_type(fn, "x", x.dtype)
    return code, px, ldx, None, _lib.qmm_w8a8_workspace_bytes(x.shape[0], x.shape[1], code)


def w8a8_gemm(x, W, sw, sx=None, out=None, out_dtype=torch.float32):
    """y (M, N) = sx[m] sw[n] sum_k xq[m, k] W[n, k], W (N, K) int8 and sw (N,)
    float32.  x is (M, K) int8 codes with scales sx, or float values that the
    call quantizes as quantize_tokens does.  y is `out`, else a new tensor of
    out_dtype (float32, float16, bfloat16)."""
    fn = "qmm_w8a8_gemm"
    code, px, ldx, ps, need = _left(fn, x, sx)
    M, K = x.shape
    pw, ldw = _int8_matrix(fn, "W", W)
    N = W.shape[0]
    if W.shape[1] != K:
        _refuse(fn, f"W must be (N, {K}), got {tuple(W.shape)}")
    psw = _scale(fn, "sw", sw, N)
    index = _one_gpu(fn, x, sx, W, sw, out)
    y, ycode, py, ldy = _output(fn, "out", out, out_dtype, (M, N), x.device)
    ws = torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
    _run(index, lambda st: _lib.qmm_w8a8_gemm(px, code, ldx, ps, pw, ldw, psw, py, ycode, ldy, M, N,
                                              K, ws.data_ptr() if need else None, need, st))
    return y


def _pair(fn, Wg, sg, Wu, su, K):
    pg, ldw = _int8_matrix(fn, "Wg", Wg)
    N = Wg.shape[0]
    if Wg.shape[1] != K:
        _refuse(fn, f"Wg must be (N, {K}), got {tuple(Wg.shape)}")
    pu, ldu = _int8_matrix(fn, "Wu", Wu, (N, K))
    if ldu != ldw:
        _refuse(fn, f"Wg and Wu must have the same row stride (got {ldw} and {ldu})")
    return N, pg, pu, ldw, _scale(fn, "sg", sg, N), _scale(fn, "su", su, N)


def w8a8_gated(x, Wg, sg, Wu, su, act="silu", sx=None, out=None, out_dtype=torch.float32):
    """h (M, N) = act(g) * u, with g and u the products of w8a8_gemm with Wg and
    Wu (N, K), in one pass; act is "silu", "gelu" (by erf) or "gelu_tanh".  x,
    sx, out and out_dtype as for w8a8_gemm."""
    fn = "qmm_w8a8_gated"
    a = _act(fn, act)
    code, px, ldx, ps, need = _left(fn, x, sx)
    M, K = x.shape
    N, pg, pu, ldw, psg, psu = _pair(fn, Wg, sg, Wu, su, K)
    index = _one_gpu(fn, x, sx, Wg, sg, Wu, su, out)
    h, hcode, ph, ldh = _output(fn, "out", out, out_dtype, (M, N), x.device)
    ws = torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
    _run(index, lambda st: _lib.qmm_w8a8_gated(px, code, ldx, ps, pg, psg, pu, psu, ldw, ph, hcode,
                                               ldh, M, N, K, a, ws.data_ptr() if need else None,
                                               need, st))
    return h


_GRADS = {torch.float16: QMM_F16, torch.bfloat16: QMM_BF16}


def w8a8_gemm_backward(dy, xq, sx, W, sw, weight_grad=True):
    """(dx (M, K), dW (N, K) or None) of dy's type (float16, bfloat16): the
    gradients of w8a8_gemm with respect to the dequantized activations sx xq
    and weights sw W.  Without weight_grad, xq and sx may be None."""
    fn = "qmm_w8a8_gemm_backward"
    pd, ldd = _matrix(fn, "dy", dy)
    code = _float_type(fn, "dy", dy.dtype, _GRADS)
    M, N = dy.shape
    pw, ldw = _int8_matrix(fn, "W", W)
    K = W.shape[1]
    if W.shape[0] != N:
        _refuse(fn, f"W must be ({N}, K), got {tuple(W.shape)}")
    psw = _scale(fn, "sw", sw, N)
    px, ldx, ps = None, 0, None
    if weight_grad:
        px, ldx = _int8_matrix(fn, "xq", xq, (M, K))
        ps = _scale(fn, "sx", sx, M)
    index = _one_gpu(fn, dy, W, sw, *((xq, sx) if weight_grad else ()))
    dx = torch.empty((M, K), dtype=dy.dtype, device=dy.device)
    dw = torch.empty((N, K), dtype=dy.dtype, device=dy.device) if weight_grad else None
    need = _lib.qmm_w8a8_backward_workspace_bytes(M, N, K, 0, int(weight_grad))
    ws = torch.empty(need, dtype=torch.uint8, device=dy.device)
    ld = max(K, 1)
    _run(index, lambda st: _lib.qmm_w8a8_gemm_backward(
        pd, code, ldd, px, ldx, ps, pw, ldw, psw, dx.data_ptr(), ld,
        dw.data_ptr() if weight_grad else None, ld, M, N, K, ws.data_ptr(), need, st))
    return dx, dw


def w8a8_gated_backward(dh, xq, sx, Wg, sg, Wu, su, act="silu", weight_grad=True):
    """(dx (M, K), dWg (N, K) or None, dWu or None) of dh's type: the gradients
    of w8a8_gated with respect to the dequantized activations and weights.  g
    and u are made again from the codes."""
    fn = "qmm_w8a8_gated_backward"
    a = _act(fn, act)
    pd, ldd = _matrix(fn, "dh", dh)
    code = _float_type(fn, "dh", dh.dtype, _GRADS)
    px, ldx = _int8_matrix(fn, "xq", xq)
    M, K = xq.shape
    N, pg, pu, ldw, psg, psu = _pair(fn, Wg, sg, Wu, su, K)
    if dh.shape != (M, N):
        _refuse(fn, f"dh must be {(M, N)}, got {tuple(dh.shape)}")
    ps = _scale(fn, "sx", sx, M)
    index = _one_gpu(fn, dh, xq, sx, Wg, sg, Wu, su)
    new = lambda rows: torch.empty((rows, K), dtype=dh.dtype, device=dh.device)  # noqa: E731
    dx = new(M)
    dwg, dwu = (new(N), new(N)) if weight_grad else (None, None)
    need = _lib.qmm_w8a8_backward_workspace_bytes(M, N, K, 1, int(weight_grad))
    ws = torch.empty(need, dtype=torch.uint8, device=dh.device)
    ld = max(K, 1)
    _run(index, lambda st: _lib.qmm_w8a8_gated_backward(
        pd, code, ldd, px, ldx, ps, pg, psg, pu, psu, ldw, dx.data_ptr(), ld,
        dwg.data_ptr() if weight_grad else None, dwu.data_ptr() if weight_grad else None, ld, M, N,
        K, a, ws.data_ptr(), need, st))
    return dx, dwg, dwu
