"""The int8 x int8 entry points refuse what they cannot take, before any HIP
call (CPU only: every call below fails its checks or has nothing to do), and
the 64-bit references of the GPU tests agree with worked examples and
differences."""
import ctypes
import math
import os
import re

import pytest
import torch

import int8_util as u8

qmm = pytest.importorskip("gemv_only_quant_amd")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, MIS = 0x10000, 0x10004  # addresses that never reach a kernel
ARG, UNS = qmm.QMM_ERR_ARG, qmm.QMM_ERR_UNSUPPORTED
L = qmm._lib


def test_exports_every_declared_symbol():
    src = open(os.path.join(ROOT, "include", "qmm_int8.h")).read()
    names = set(re.findall(r"QMM_API\s+[\w\s\*]+?\b(qmm_\w+)\s*\(", src))
    assert names == set(qmm.EXPORTS_INT8)
    lib = ctypes.CDLL(qmm.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n


def gemm(**o):
    a = dict(x=A, t=3, ldx=64, sx=A, W=A, ldw=64, sw=A, y=A, yt=2, ldy=32, M=4, N=32, K=64, ws=None, n=0)
    a.update(o)
    return L.qmm_w8a8_gemm(a["x"], a["t"], a["ldx"], a["sx"], a["W"], a["ldw"], a["sw"], a["y"], a["yt"],
                           a["ldy"], a["M"], a["N"], a["K"], a["ws"], a["n"], 0)


def gated(**o):
    a = dict(x=A, t=3, ldx=64, sx=A, Wg=A, sg=A, Wu=A, su=A, ldw=64, h=A, ht=2, ldh=32, M=4, N=32, K=64,
             act=0, ws=None, n=0)
    a.update(o)
    return L.qmm_w8a8_gated(a["x"], a["t"], a["ldx"], a["sx"], a["Wg"], a["sg"], a["Wu"], a["su"],
                            a["ldw"], a["h"], a["ht"], a["ldh"], a["M"], a["N"], a["K"], a["act"],
                            a["ws"], a["n"], 0)


def gemm_bwd(**o):
    a = dict(dy=A, t=1, lddy=32, x=A, ldx=64, sx=A, W=A, ldw=64, sw=A, dx=A, lddx=64, dW=A, lddw=64, M=4,
             N=32, K=64, ws=A, n=1 << 30)
    a.update(o)
    return L.qmm_w8a8_gemm_backward(a["dy"], a["t"], a["lddy"], a["x"], a["ldx"], a["sx"], a["W"],
                                    a["ldw"], a["sw"], a["dx"], a["lddx"], a["dW"], a["lddw"], a["M"],
                                    a["N"], a["K"], a["ws"], a["n"], 0)


def gated_bwd(**o):
    a = dict(dh=A, t=1, lddh=32, x=A, ldx=64, sx=A, Wg=A, sg=A, Wu=A, su=A, ldw=64, dx=A, lddx=64, dWg=A,
             dWu=A, lddw=64, M=4, N=32, K=64, act=0, ws=A, n=1 << 30)
    a.update(o)
    return L.qmm_w8a8_gated_backward(a["dh"], a["t"], a["lddh"], a["x"], a["ldx"], a["sx"], a["Wg"],
                                     a["sg"], a["Wu"], a["su"], a["ldw"], a["dx"], a["lddx"], a["dWg"],
                                     a["dWu"], a["lddw"], a["M"], a["N"], a["K"], a["act"], a["ws"],
                                     a["n"], 0)


def quant(**o):
    a = dict(x=A, t=0, ldx=64, q=A, ldq=64, s=A, M=4, K=64)
    a.update(o)
    return L.qmm_quantize_tokens(a["x"], a["t"], a["ldx"], a["q"], a["ldq"], a["s"], a["M"], a["K"], 0)


BAD = [
    (quant, dict(t=3), ARG, "x_dtype"), (quant, dict(M=-1), ARG, "negative"),
    (quant, dict(x=None), ARG, "NULL x"), (quant, dict(s=None), ARG, "NULL sx"),
    (quant, dict(ldx=63), ARG, "leading dimension of x"), (quant, dict(x=A + 1), ARG, "aligned to its elements"),
    (quant, dict(K=60, ldq=60), UNS, "multiple of 16"), (quant, dict(q=MIS), ARG, "16-byte"),
    (quant, dict(K=1 << 17, ldx=1 << 17, ldq=1 << 17), UNS, "too large"),
    (gemm, dict(t=4), ARG, "x_dtype"), (gemm, dict(yt=3), ARG, "output type"),
    (gemm, dict(K=-1), ARG, "negative"), (gemm, dict(K=1 << 17, ldx=1 << 17, ldw=1 << 17), UNS, "exact 32-bit"),
    (gemm, dict(sx=None), ARG, "NULL sx"), (gemm, dict(x=None), ARG, "NULL x"),
    (gemm, dict(t=1), ARG, "must be NULL for values"), (gemm, dict(t=1, sx=None), ARG, "workspace of"),
    (gemm, dict(t=1, sx=None, ws=MIS, n=1 << 20), ARG, "16-byte aligned"),
    (gemm, dict(t=1, sx=None, ws=A, n=100), ARG, "workspace of"),
    (gemm, dict(W=MIS), ARG, "16-byte"), (gemm, dict(ldw=72), UNS, "multiple of 16"),
    (gemm, dict(ldw=48), ARG, "leading dimension of W"), (gemm, dict(ldx=1 << 22), UNS, "too large"),
    (gemm, dict(sw=None), ARG, "NULL sw"), (gemm, dict(y=None), ARG, "NULL y"),
    (gemm, dict(ldy=31), ARG, "leading dimension of y"), (gemm, dict(y=A + 2), ARG, "aligned to its elements"),
    (gated, dict(act=3), ARG, "act must be"), (gated, dict(act=-1), ARG, "act must be"),
    (gated, dict(Wu=None), ARG, "NULL Wu"), (gated, dict(su=None), ARG, "NULL su"),
    (gated, dict(sg=MIS + 1), ARG, "4-byte"), (gated, dict(h=None), ARG, "NULL h"),
    (gemm_bwd, dict(t=2), ARG, "dtype"), (gemm_bwd, dict(dx=None), ARG, "NULL dx"),
    (gemm_bwd, dict(x=None), ARG, "NULL xq"), (gemm_bwd, dict(sx=None), ARG, "NULL sx"),
    (gemm_bwd, dict(dy=None), ARG, "NULL dy"), (gemm_bwd, dict(lddx=63), ARG, "leading dimension of dx"),
    (gemm_bwd, dict(lddw=63), ARG, "leading dimension of dW"), (gemm_bwd, dict(ws=None), ARG, "workspace of"),
    (gemm_bwd, dict(n=1000), ARG, "workspace of"), (gemm_bwd, dict(ws=A + 16), ARG, "256-byte"),
    (gemm_bwd, dict(N=1 << 21, lddy=1 << 21), UNS, "too large"), (gemm_bwd, dict(M=1 << 21), UNS, "too large"),
    (gated_bwd, dict(act=9), ARG, "act must be"), (gated_bwd, dict(dWu=None), ARG, "together"),
    (gated_bwd, dict(dWg=None), ARG, "together"), (gated_bwd, dict(x=None), ARG, "NULL xq"),
    (gated_bwd, dict(x=None, dWg=None, dWu=None), ARG, "NULL xq"), (gated_bwd, dict(dh=None), ARG, "NULL dh"),
    (gated_bwd, dict(t=3), ARG, "dtype"),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_refused(i):
    fn, over, status, text = BAD[i]
    assert fn(**over) == status
    assert text in qmm.qmm_last_error(), qmm.qmm_last_error()


@pytest.mark.parametrize("fn,over", [(quant, dict(M=0, x=None, q=None, s=None)), (gemm, dict(M=0, x=None, y=None)),
                                     (gemm, dict(N=0, W=None, y=None)), (gated, dict(M=0)), (gemm_bwd, dict(K=0)),
                                     (gemm_bwd, dict(M=0, dW=None)), (gemm_bwd, dict(M=0, N=0)),
                                     (gated_bwd, dict(M=0, dWg=None, dWu=None))])
def test_nothing_to_do(fn, over):
    assert fn(**over) == qmm.QMM_OK and qmm.qmm_last_error() == ""


def test_workspace_sizes():
    assert L.qmm_w8a8_workspace_bytes(3, 100, 1) == 3 * 112 + 12
    assert L.qmm_w8a8_workspace_bytes(3, 4096, 1) == 0  # a few tokens: quantized within the launch
    assert L.qmm_w8a8_workspace_bytes(5, 4096, 1) == 5 * 4096 + 20
    assert L.qmm_w8a8_workspace_bytes(3, 100, 3) == 0 and L.qmm_w8a8_workspace_bytes(0, 100, 1) == 0
    assert L.qmm_w8a8_workspace_bytes(3, 1 << 17, 1) == 0
    need = L.qmm_w8a8_backward_workspace_bytes
    assert need(0, 5, 5, 0, 0) == 0 and need(5, 5, 1 << 17, 0, 0) == 0
    assert 0 < need(100, 200, 300, 0, 0) < need(100, 200, 300, 0, 1) < need(100, 200, 300, 1, 1)


@pytest.mark.parametrize("fn,over", [(quant, dict(M=2 ** 31 - 1024)), (gemm, dict(M=2 ** 31 - 1024)),
                                     (gemm, dict(N=2 ** 31 - 1, ldy=1 << 21)), (gated, dict(M=2 ** 31 - 1)),
                                     (gated_bwd, dict(N=1 << 20, lddh=1 << 20))])
def test_sizes_whose_indices_leave_their_types(fn, over):
    assert fn(**over) == UNS and "too large" in qmm.qmm_last_error()


def test_no_workspace_for_sizes_that_are_refused():
    assert L.qmm_w8a8_workspace_bytes(2 ** 31 - 1024, 64, 1) == 0
    need = L.qmm_w8a8_backward_workspace_bytes
    assert need(1 << 21, 8, 8, 0, 0) == 0 and need(8, 1 << 20, 8, 1, 0) == 0 < need(8, 1 << 20, 8, 0, 0)


def raises(fn, text, status=ARG):
    with pytest.raises(qmm.QmmError) as e:
        fn()
    assert text in str(e.value) and e.value.status == status, str(e.value)


def test_binding_checks():
    x, w, s = torch.zeros(4, 64), torch.zeros((32, 64), dtype=torch.int8), torch.zeros(32)
    q, sx = torch.zeros((4, 64), dtype=torch.int8), torch.zeros(4)
    d = torch.zeros((4, 32), dtype=torch.float16)
    raises(lambda: qmm.w8a8_gemm(x, w, s), "GPU tensors")
    raises(lambda: qmm.w8a8_gemm(x.double(), w, s), "x must be one of")
    raises(lambda: qmm.w8a8_gemm(q, w, s), "needs its scales")
    raises(lambda: qmm.w8a8_gemm(x, w, s, sx=sx), "goes with int8")
    raises(lambda: qmm.w8a8_gemm(x, w.int(), s), "W must be int8")
    raises(lambda: qmm.w8a8_gemm(x, w[:, :32], s), "W must be (N, 64)")
    raises(lambda: qmm.w8a8_gemm(x[0], w, s), "2-D")
    raises(lambda: qmm.w8a8_gemm(x, w.t().contiguous().t(), s), "unit column stride")
    raises(lambda: qmm.w8a8_gemm(x, w, s[:31]), "sw must hold 32")
    raises(lambda: qmm.w8a8_gemm(x, w, s.half()), "sw must be a float32")
    raises(lambda: qmm.w8a8_gemm(x[:, :60], torch.zeros((32, 60), dtype=torch.int8), s),
           "whole 16 bytes", UNS)
    raises(lambda: qmm.w8a8_gated(x, w, s, w, s, act="relu"), "act must be one of")
    raises(lambda: qmm.w8a8_gated(x, w, s, w[:16], s), "Wu must be")
    raises(lambda: qmm.w8a8_gated(x, w, s, torch.zeros((32, 80), dtype=torch.int8)[:, :64], s), "same row stride")
    raises(lambda: qmm.w8a8_gemm_backward(d.float(), q, sx, w, s), "dy must be one of")
    raises(lambda: qmm.w8a8_gemm_backward(d, q[:3], sx, w, s), "xq must be")
    raises(lambda: qmm.w8a8_gemm_backward(d[:, :5], q, sx, w, s), "W must be (5, K)")
    raises(lambda: qmm.w8a8_gated_backward(d[:3], q, sx, w, s, w, s), "dh must be")
    raises(lambda: qmm.w8a8_gated_backward(d, q, sx[:3], w, s, w, s), "sx must hold 4")
    raises(lambda: qmm.quantize_tokens(x.int()), "x must be one of")
    raises(lambda: qmm.quantize_tokens(x), "GPU tensors")


def test_quantizer_reference_worked_example():
    # scale 127 / 127 = 1: codes are the values rounded to nearest even
    x = torch.tensor([[127.0, 0.5, 1.5, -0.5, -2.5, 3.49, -3.51, 0.0], [0.0] * 8])
    q, s = u8.quantize_ref(x)
    assert s.tolist() == [1.0, 0.0]
    assert q.tolist() == [[127, 0, 2, 0, -2, 3, -4, 0], [0] * 8]


@pytest.mark.parametrize("act", qmm.ACTIVATIONS)
def test_gradient_reference_against_differences(act):
    """The formulas of the gradients against central differences of the forward
    formula, in 64 bits: eps 1e-5 leaves eps^2 of the third derivative and
    1e-16 / eps of rounding, both below 1e-9 of the terms' size."""
    m, n, k = 7, 9, 11
    q, sx = u8.quantize_ref(u8.tokens(m, k, seed=1))
    (wg, sg), (wu, su) = u8.weight(n, k, seed=2), u8.weight(n, k, seed=3)
    dh = torch.randn((m, n), generator=torch.Generator().manual_seed(4)).double()
    ref = u8.gated_backward_ref(act, dh, q, sx, wg, sg, wu, su)
    xh = q.double() * sx.double()[:, None]
    gh, uh = wg.double() * sg.double()[:, None], wu.double() * su.double()[:, None]

    def loss(x, g, u):
        return (u8.act_ref(act, x @ g.t())[0] * (x @ u.t()) * dh).sum()

    for i, r in enumerate(ref):
        v = torch.randn(r.shape, generator=torch.Generator().manual_seed(5 + i)).double()
        at = lambda e: [t + (e * v if j == i else 0) for j, t in enumerate((xh, gh, uh))]  # noqa: E731
        want = (loss(*at(1e-5)) - loss(*at(-1e-5))) / 2e-5
        assert math.isclose(float((r * v).sum()), float(want), rel_tol=1e-7, abs_tol=1e-7)
