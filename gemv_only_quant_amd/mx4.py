"""Python binding of the microscaled 4-bit operators (include/qmm_mx4.h): the
quantizer and its inverse, the offline layout of weights, the product, and a
mixture-of-experts layer for a few tokens.

    q, s = mx4_quantize(x)                       # (M, K) -> codes (M, 16 B), scales (M, B), B = ceil(K / 32)
    x = mx4_dequantize(q, s, K)
    W = mx4_pack(*mx4_quantize(w))               # (N, K) weights, laid out once; (E, N, ..) for experts
    y = mx4_gemm(x, W, N)                        # x values, quantized by the call
    y = mx4_gemm(q, W, N, sx=s)                  # or codes with their scales
    y = mx4_moe(x, Wg, Wu, Wd, I, logits=r, top_k=8)          # sum_j w_j Wd_e (act(Wg_e x) * (Wu_e x))
    y = mx4_moe(x, Wg, Wu, Wd, I, ids=i, weights=w)           # or experts already chosen

Matrices are 2-D tensors with unit column stride (a slice of the columns of a
wider tensor will do).  Codes are uint8, two values to a byte, the earlier in the
low half; scales are uint8, 2^(byte - 127).  All of a call's tensors sit on one
GPU; the work goes to that GPU's current stream and the scratch comes from torch's
allocator on that stream, so tensors in use on another stream need the usual
wait_stream or record_stream.  Nothing here is an autograd function: a call whose
operands require gradients warns that it passes none on, unless gradients are off.
"""
import ctypes

import torch

from . import _check, _lib
from .int8 import _INT_MAX, _act, _float_type, _matrix, _one_gpu, _output, _refuse

QMM_MX4 = 4  # x_dtype of activations that are codes already
QMM_MX4_MAX_TOKENS, QMM_MX4_MAX_TOP_K, QMM_MX4_MAX_EXPERTS = 64, 32, 1024

_P, _I, _L, _S = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
_lib.qmm_mx4_quantize.argtypes = [_P, _I, _L, _P, _L, _P, _L, _I, _I, _P]
_lib.qmm_mx4_dequantize.argtypes = [_P, _L, _P, _L, _P, _I, _L, _I, _I, _P]
_lib.qmm_mx4_packed_bytes.argtypes = [_I, _I]
_lib.qmm_mx4_packed_bytes.restype = _S
_lib.qmm_mx4_pack.argtypes = [_P, _L, _P, _L, _P, _I, _I, _I, _P]
_lib.qmm_mx4_workspace_bytes.argtypes = [_I, _I, _I]
_lib.qmm_mx4_workspace_bytes.restype = _S
_lib.qmm_mx4_gemm.argtypes = [_P, _I, _L, _P, _L, _P, _P, _I, _L, _I, _I, _I, _P, _S, _P]
_lib.qmm_mx4_moe_workspace_bytes.argtypes = [_I] * 7
_lib.qmm_mx4_moe_workspace_bytes.restype = _S
_lib.qmm_mx4_moe.argtypes = [_P, _I, _L, _P, _P, _P, _P, _I, _L, _I, _I, _I, _I, _I, _I, _P, _I, _L, _I, _P,
                             _I, _P, _I, _P, _S, _P]

EXPORTS_MX4 = ("qmm_mx4_quantize", "qmm_mx4_dequantize", "qmm_mx4_packed_bytes", "qmm_mx4_pack",
               "qmm_mx4_workspace_bytes", "qmm_mx4_gemm", "qmm_mx4_moe_workspace_bytes", "qmm_mx4_moe")

# the current GPU, and its current stream's handle without the object around it (a microsecond less for each call)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run(index, call, *args):
    """call(*args, stream) with the GPU current, on its current stream."""
    if index == _device():
        _check(call(*args, _raw_stream(index)))
    else:
        with torch.cuda.device(index):
            _check(call(*args, _raw_stream(index)))


def _size(fn, name, v):
    """A size that is no tensor's: an int that the library's would not cut off."""
    if not isinstance(v, int) or not 0 <= v <= _INT_MAX:
        _refuse(fn, f"{name} must be a size below 2^31, got {v!r}")


def _blocks(K):
    return -(-K // 32)


def _values(B):
    """Values of rows of B blocks of codes: all of them count, but the library's sizes end at 2^20 - 1, whose
    last block is whole too."""
    return 32 * B - (B == 1 << 15)


def _bytes_matrix(fn, name, t, shape=None):
    """As _matrix, for bytes."""
    if isinstance(t, torch.Tensor) and t.dtype != torch.uint8:
        _refuse(fn, f"{name} must be uint8, got {t.dtype}")
    return _matrix(fn, name, t, shape)


def _coded(fn, codes, scales):
    """(pointer, ld) of codes and of scales, and the number of blocks."""
    pc, ldc = _bytes_matrix(fn, "codes", codes)
    rows, cols = codes.shape
    if cols % 16:
        _refuse(fn, f"codes have rows of whole blocks, 16 bytes each (got {cols})")
    ps, lds = _bytes_matrix(fn, "scales", scales, (rows, cols // 16))
    return pc, ldc, ps, lds, cols // 16


def _result(fn, like, out, out_dtype, shape):
    """As _output, a new tensor from another of its GPU (half a microsecond less)."""
    if out is not None:
        return _output(fn, "out", out, out_dtype, shape, like.device)
    code = _float_type(fn, "out_dtype", out_dtype)
    out = like.new_empty(shape, dtype=out_dtype)
    return out, code, out.data_ptr(), max(shape[1], 1)


def _packed(fn, name, W, need):
    """Pointer of a packed weight of `need` bytes."""
    if not isinstance(W, torch.Tensor) or W.dtype != torch.uint8:
        _refuse(fn, f"{name} must be a uint8 tensor")
    if W.numel() != need or not W.is_contiguous():
        _refuse(fn, f"{name} must hold {need} contiguous bytes (got {tuple(W.shape)}); mx4_pack makes it")
    return W.data_ptr()


def mx4_quantize(x):
    """x (M, K) float32 / float16 / bfloat16 -> (codes (M, 16 B), scales (M, B)) uint8, B = ceil(K / 32).
    The scales are a view of rows padded to 4 bytes."""
    fn = "qmm_mx4_quantize"
    px, ldx = _matrix(fn, "x", x)
    code = _float_type(fn, "x", x.dtype)
    index = _one_gpu(fn, x)
    M, K = x.shape
    B = _blocks(K)
    q = x.new_empty((M, 16 * B), dtype=torch.uint8)
    lds = max(4, -(-B // 4) * 4)
    s = x.new_empty((M, lds), dtype=torch.uint8)
    _run(index, _lib.qmm_mx4_quantize, px, code, ldx, q.data_ptr(), max(16 * B, 16), s.data_ptr(), lds,
         M, K)
    return q, s if lds == B else s[:, :B]


def mx4_dequantize(codes, scales, K=None, out=None, out_dtype=torch.float32):
    """The values (M, K) that codes (M, 16 B) and scales (M, B) stand for; K is 32 B, or less where the last
    block is not whole.  They go to `out`, else to a new tensor of out_dtype."""
    fn = "qmm_mx4_dequantize"
    pc, ldc, ps, lds, B = _coded(fn, codes, scales)
    K = 32 * B if K is None else K
    _size(fn, "K", K)
    if _blocks(K) != B:
        _refuse(fn, f"K={K} does not have {B} blocks of 32")
    index = _one_gpu(fn, codes, scales, out)
    M = codes.shape[0]
    y, code, py, ldy = _result(fn, codes, out, out_dtype, (M, K))
    _run(index, _lib.qmm_mx4_dequantize, pc, ldc, ps, lds, py, code, ldy, M, K)
    return y


def mx4_packed_bytes(N, K):
    """Bytes of a packed weight (N, K); 0 for sizes that there cannot be."""
    if not (0 <= N <= _INT_MAX and 0 <= K <= _INT_MAX):
        return 0
    return _lib.qmm_mx4_packed_bytes(N, K)


def mx4_pack(codes, scales):
    """A weight's codes (N, 16 B) and scales (N, B), as mx4_quantize gives them, to the layout that the products
    read (uint8, one dimension); codes (E, N, 16 B) and scales (E, N, B) of E experts to (E, bytes)."""
    fn = "qmm_mx4_pack"
    for name, t in (("codes", codes), ("scales", scales)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8:
            _refuse(fn, f"{name} must be a uint8 tensor")
    batch = ()
    if codes.dim() == 3 and scales.dim() == 3:
        batch = (codes.shape[0],)
        if scales.shape[:2] != codes.shape[:2]:
            _refuse(fn, f"scales must be {(*codes.shape[:2], codes.shape[2] // 16)}, got {tuple(scales.shape)}")
        N = codes.shape[1]
        codes, scales = codes.flatten(0, 1), scales.flatten(0, 1)
    elif codes.dim() == 2:
        N = codes.shape[0]
    else:
        _refuse(fn, "codes and scales must both be 2-D, or both 3-D")
    pc, ldc, ps, lds, B = _coded(fn, codes, scales)
    index = _one_gpu(fn, codes, scales)
    E = batch[0] if batch else 1
    W = torch.empty((*batch, mx4_packed_bytes(N, _values(B))), dtype=torch.uint8, device=codes.device)
    _run(index, _lib.qmm_mx4_pack, pc, ldc, ps, lds, W.data_ptr(), E, N, _values(B))
    return W


def mx4_gemm(x, W, N, sx=None, out=None, out_dtype=torch.float32):
    """y (M, N) = x^ W^t, W a weight (N, K) packed by mx4_pack.  x is (M, 16 B) uint8 codes with scales sx (M,
    B), or (M, K) float values that the call quantizes as mx4_quantize does.  y is `out`, else a new tensor of
    out_dtype (float32, float16, bfloat16)."""
    fn = "qmm_mx4_gemm"
    _size(fn, "N", N)
    ps, lds = None, 0
    if isinstance(x, torch.Tensor) and x.dtype == torch.uint8:
        if sx is None:
            _refuse(fn, "uint8 x needs its scales (sx)")
        px, ldx, ps, lds, B = _coded(fn, x, sx)
        code, K = QMM_MX4, _values(B)
    else:
        px, ldx = _matrix(fn, "x", x)
        if sx is not None:
            _refuse(fn, "sx goes with uint8 x")
        code = _float_type(fn, "x", x.dtype)
        K = x.shape[1]
    M = x.shape[0]
    need = _lib.qmm_mx4_workspace_bytes(M, K, code)
    pw = _packed(fn, "W", W, mx4_packed_bytes(N, K))
    index = _one_gpu(fn, x, sx, W, out)
    y, ycode, py, ldy = _result(fn, x, out, out_dtype, (M, N))
    ws = x.new_empty(need, dtype=torch.uint8) if need else None
    _run(index, _lib.qmm_mx4_gemm, px, code, ldx, ps, lds, pw, py, ycode, ldy, M, N, K,
         ws.data_ptr() if need else None, need)
    return y


def mx4_moe(x, Wg, Wu, Wd, I, logits=None, top_k=None, renormalize=True, ids=None, weights=None, act="silu",
            out=None, out_dtype=torch.float32):
    """y (T, D) = sum_j w[t, j] Wd_e (act(Wg_e x[t]) * (Wu_e x[t])), e = ids[t, j], for up to 64 tokens x (T, D).
    Wg and Wu are E packed weights (I, D), Wd E packed weights (D, I), each (E, bytes) as mx4_pack makes it.
    The experts are the top_k largest of logits (T, E), weighted by the softmax over them (renormalize) or over
    all; or ids (T, k) int32 / int64 with weights (T, k): an id outside [0, E) counts for nothing.  Activations
    are not quantized, and what lies between the halves is fp32.  y is `out`, else a new tensor of out_dtype."""
    fn = "qmm_mx4_moe"
    _size(fn, "I", I)
    a = _act(fn, act)
    px, ldx = _matrix(fn, "x", x)
    xcode = _float_type(fn, "x", x.dtype)
    T, D = x.shape
    if not isinstance(Wg, torch.Tensor) or Wg.dim() != 2:
        _refuse(fn, "Wg must be (E, bytes) uint8")
    E = Wg.shape[0]
    up, down = mx4_packed_bytes(I, D), mx4_packed_bytes(D, I)
    pg, pu, pd = _packed(fn, "Wg", Wg, E * up), _packed(fn, "Wu", Wu, E * up), _packed(fn, "Wd", Wd, E * down)
    pl, lcode, ldl, pi, isize, pw, wcode = None, 0, 0, None, 0, None, 0
    if logits is not None:
        if ids is not None or weights is not None:
            _refuse(fn, "logits, or ids and weights, not both")
        if top_k is None:
            _refuse(fn, "logits need top_k")
        _size(fn, "top_k", top_k)
        pl, ldl = _matrix(fn, "logits", logits, (T, E))
        lcode = _float_type(fn, "logits", logits.dtype)
        k = top_k
    else:
        if ids is None or weights is None:
            _refuse(fn, "logits and top_k, or ids and weights, must be given")
        for name, t in (("ids", ids), ("weights", weights)):
            if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.shape[0] != T or not t.is_contiguous():
                _refuse(fn, f"{name} must be a contiguous ({T}, k) tensor")
        if ids.dtype not in (torch.int32, torch.int64):
            _refuse(fn, f"ids must be int32 or int64, got {ids.dtype}")
        if weights.shape != ids.shape:
            _refuse(fn, f"weights must be {tuple(ids.shape)}, got {tuple(weights.shape)}")
        k = ids.shape[1]
        if top_k is not None and top_k != k:
            _refuse(fn, f"top_k={top_k}, but ids has {k} a token")
        pi, isize, pw, wcode = ids.data_ptr(), ids.element_size(), weights.data_ptr(), \
            _float_type(fn, "weights", weights.dtype)
    index = _one_gpu(fn, x, Wg, Wu, Wd, logits, ids, weights, out)
    y, ycode, py, ldy = _result(fn, x, out, out_dtype, (T, D))
    need = _lib.qmm_mx4_moe_workspace_bytes(T, D, I, E, k, xcode, ycode)
    ws = x.new_empty(need, dtype=torch.uint8) if need else None
    _run(index, _lib.qmm_mx4_moe, px, xcode, ldx, pg, pu, pd, py, ycode, ldy, T, D, I, E, k, a, pl, lcode, ldl,
         int(bool(renormalize)), pi, isize, pw, wcode, ws.data_ptr() if need else None, need)
    return y
