"""The microscaled 4-bit entry points refuse what they cannot take, before any
HIP call (CPU only: every call below fails its checks or has nothing to do), and
the 64-bit references of the GPU tests agree with worked examples."""
import ctypes
import math
import os
import re

import pytest
import torch

import mx4_util as m4

qmm = pytest.importorskip("gemv_only_quant_amd")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, MIS = 0x10000, 0x10004  # addresses that never reach a kernel
ARG, UNS = qmm.QMM_ERR_ARG, qmm.QMM_ERR_UNSUPPORTED
L = qmm._lib


def test_exports_every_declared_symbol():
    src = open(os.path.join(ROOT, "include", "qmm_mx4.h")).read()
    names = set(re.findall(r"QMM_API\s+[\w\s\*]+?\b(qmm_\w+)\s*\(", src))
    assert names == set(qmm.EXPORTS_MX4)
    lib = ctypes.CDLL(qmm.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n


def call(name, **defaults):
    def f(**over):
        a = {**defaults, **over}
        assert a.keys() == defaults.keys()
        return getattr(L, name)(*a.values(), 0)
    return f


quant = call("qmm_mx4_quantize", x=A, t=1, ldx=64, q=A, ldq=32, s=A, lds=4, M=4, K=64)
dequant = call("qmm_mx4_dequantize", q=A, ldq=32, s=A, lds=2, y=A, t=2, ldy=64, M=4, K=64)
packw = call("qmm_mx4_pack", q=A, ldq=32, s=A, lds=2, W=A, batch=2, N=32, K=64)
gemm = call("qmm_mx4_gemm", x=A, t=4, ldx=32, sx=A, ldsx=4, W=A, y=A, yt=2, ldy=32, M=4, N=32, K=64, ws=None, n=0)
moe = call("qmm_mx4_moe", x=A, t=1, ldx=64, Wg=A, Wu=A, Wd=A, y=A, yt=2, ldy=64, T=4, D=64, I=32, E=8, k=2, act=0,
           lg=A, lt=2, ldl=8, norm=1, ids=None, isz=0, w=None, wt=0, ws=A, n=1 << 30)
given = dict(lg=None, ids=A, isz=4, w=A, wt=2)

BAD = [
    (quant, dict(t=3), ARG, "x_dtype"), (quant, dict(M=-1), ARG, "negative"), (quant, dict(x=None), ARG, "NULL x"),
    (quant, dict(q=None), ARG, "NULL codes"), (quant, dict(s=None), ARG, "NULL scales"),
    (quant, dict(ldx=63), ARG, "leading dimension of x"), (quant, dict(x=A + 1), ARG, "2-byte"),
    (quant, dict(ldq=16), ARG, "leading dimension of codes"), (quant, dict(ldq=40), UNS, "multiple of 16"),
    (quant, dict(q=MIS), ARG, "16-byte"), (quant, dict(lds=1), ARG, "leading dimension of scales"),
    (quant, dict(K=1 << 20), UNS, "too large"), (quant, dict(M=2 ** 31 - 1), UNS, "too large"),
    (quant, dict(ldx=1 << 22), UNS, "too large"),
    (dequant, dict(t=4), ARG, "y_dtype"), (dequant, dict(K=-1), ARG, "negative"), (dequant, dict(y=None), ARG, "NULL y"),
    (dequant, dict(ldq=31), ARG, "leading dimension of codes"), (dequant, dict(lds=1), ARG, "scales"),
    (dequant, dict(y=A + 2), ARG, "4-byte"), (dequant, dict(q=None), ARG, "NULL codes"),
    (packw, dict(batch=-1), ARG, "batch"), (packw, dict(W=None), ARG, "NULL W"), (packw, dict(W=MIS), ARG, "16-byte"),
    (packw, dict(ldq=16), ARG, "codes"), (packw, dict(lds=0), ARG, "scales"), (packw, dict(N=-2), ARG, "negative"),
    (packw, dict(batch=1 << 20, N=1 << 20), UNS, "too large"),
    (gemm, dict(t=3), ARG, "x_dtype"), (gemm, dict(yt=4), ARG, "y_dtype"), (gemm, dict(N=-1), ARG, "negative"),
    (gemm, dict(x=None), ARG, "NULL x"), (gemm, dict(sx=None), ARG, "NULL sx"), (gemm, dict(W=None), ARG, "NULL W"),
    (gemm, dict(W=MIS), ARG, "16-byte"), (gemm, dict(y=None), ARG, "NULL y"), (gemm, dict(ldy=31), ARG, "of y"),
    (gemm, dict(ldx=16), ARG, "of x"), (gemm, dict(ldsx=1), ARG, "of sx"), (gemm, dict(t=2, sx=None, ldx=64, x=A + 2), ARG, "4-byte"),
    (gemm, dict(t=1), ARG, "must be NULL for values"), (gemm, dict(), ARG, "workspace of"),
    (gemm, dict(t=1, sx=None, ldx=64, M=17), ARG, "workspace of"), (gemm, dict(ws=A, n=10), ARG, "workspace of"),
    (gemm, dict(ws=MIS, n=1 << 20), ARG, "16-byte aligned"),
    (gemm, dict(K=1 << 20, ldx=1 << 19, ldsx=1 << 15), UNS, "too large"), (gemm, dict(M=2 ** 31 - 1), UNS, "too large"),
    (moe, dict(t=4), ARG, "x_dtype"), (moe, dict(yt=3), ARG, "y_dtype"), (moe, dict(act=3), ARG, "act must be"),
    (moe, dict(T=-1), ARG, "negative"), (moe, dict(T=65), UNS, "too large"), (moe, dict(E=1025, ldl=1025), UNS, "too large"),
    (moe, dict(k=33, E=64, ldl=64), UNS, "too large"), (moe, dict(I=1 << 20), UNS, "too large"),
    (moe, dict(x=None), ARG, "NULL x"), (moe, dict(y=None), ARG, "NULL y"), (moe, dict(Wg=None), ARG, "NULL Wg"),
    (moe, dict(Wu=MIS), ARG, "16-byte"), (moe, dict(Wd=None), ARG, "NULL Wd"), (moe, dict(ldx=63), ARG, "of x"),
    (moe, dict(ldy=63), ARG, "of y"), (moe, dict(k=9), ARG, "top_k=9 of E=8"), (moe, dict(lt=7), ARG, "logits_dtype"),
    (moe, dict(ldl=7), ARG, "of logits"), (moe, dict(norm=2), ARG, "renormalize"), (moe, dict(ids=A), ARG, "not both"),
    (moe, dict(lg=None), ARG, "must be given"), (moe, dict(given, w=None), ARG, "must be given"),
    (moe, dict(given, ids=None), ARG, "must be given"), (moe, dict(given, isz=2), ARG, "ids_size"),
    (moe, dict(given, wt=4), ARG, "weights_dtype"), (moe, dict(given, ids=A + 4, isz=8), ARG, "aligned to their"),
    (moe, dict(ws=None), ARG, "workspace of"), (moe, dict(n=100), ARG, "workspace of"), (moe, dict(ws=A + 16), ARG, "256-byte"),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_refused(i):
    fn, over, status, text = BAD[i]
    assert fn(**over) == status, qmm.qmm_last_error()
    assert text in qmm.qmm_last_error(), qmm.qmm_last_error()


@pytest.mark.parametrize("fn,over", [
    (quant, dict(M=0, x=None, q=None, s=None)), (quant, dict(K=0, x=None, q=None, s=None)), (dequant, dict(M=0)),
    (dequant, dict(K=0)), (packw, dict(batch=0, W=None)), (packw, dict(N=0)), (packw, dict(K=0)), (gemm, dict(M=0, y=None)),
    (gemm, dict(N=0, W=None)), (moe, dict(T=0, x=None, y=None)), (moe, dict(D=0, Wd=None, ldy=1))])
def test_nothing_to_do(fn, over):
    assert fn(**over) == qmm.QMM_OK and qmm.qmm_last_error() == ""


def test_sizes():
    # strips of 16 columns, chunks of 512 values: 4096 bytes of codes and 256 of scales
    assert L.qmm_mx4_packed_bytes(16, 512) == L.qmm_mx4_packed_bytes(1, 1) == 4352
    assert L.qmm_mx4_packed_bytes(17, 512) == 2 * 4352 and L.qmm_mx4_packed_bytes(16, 513) == 2 * 4352
    assert L.qmm_mx4_packed_bytes(0, 128) == L.qmm_mx4_packed_bytes(16, 0) == L.qmm_mx4_packed_bytes(16, 1 << 20) == 0
    need = L.qmm_mx4_workspace_bytes
    assert need(0, 64, 1) == need(100, 1 << 20, 1) == need(2 ** 31 - 1, 64, 1) == need(4, 64, 3) == 0
    assert need(1, 4096, 1) == 0 and need(8, 4096, 0) == 0  # a few values: quantized within the launch
    assert need(16, 8192, 0) == need(1, 8192, 4) == 16 * 4352 and need(100, 4096, 4) == 7 * 8 * 4352
    need = L.qmm_mx4_moe_workspace_bytes
    assert need(65, 64, 64, 8, 2, 1, 1) == need(4, 64, 64, 8, 2, 4, 1) == need(0, 64, 64, 8, 2, 1, 1) == 0
    assert 0 < need(4, 64, 64, 8, 2, 1, 1) <= need(4, 64, 64, 8, 2, 2, 2)


def raises(fn, text, status=ARG):
    with pytest.raises(qmm.QmmError) as e:
        fn()
    assert text in str(e.value) and e.value.status == status, str(e.value)


@pytest.mark.parametrize("E", [1, 2, 3, 40, 1024])
def test_mixture_workspace_for_any_choice(E):
    """Given experts may be more for each token than there are."""
    need = L.qmm_mx4_moe_workspace_bytes
    for T in (1, 2, 3, 16, 63, 64):
        for k in (1, 2, 3, 8, 31, 32):
            for D, I in ((1, 1), (64, 64), (4096, 14336), (14336, 4096)):
                if T * k * max(D, I) < 1 << 27:
                    for x in (0, 1, 2):
                        assert need(T, D, I, E, k, x, x) >= 4 * T * k * (D + I)


def test_binding_checks():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    x, W = torch.zeros(4, 64), u8(qmm.mx4_packed_bytes(32, 64))
    raises(lambda: qmm.mx4_quantize(x), "GPU tensors")
    raises(lambda: qmm.mx4_quantize(x.double()), "x must be one of")
    raises(lambda: qmm.mx4_quantize(x.t()), "unit column stride")
    raises(lambda: qmm.mx4_dequantize(u8(4, 30), u8(4, 2)), "whole blocks")
    raises(lambda: qmm.mx4_dequantize(u8(4, 32), u8(4, 3)), "scales must be")
    raises(lambda: qmm.mx4_dequantize(u8(4, 32), u8(4, 2), 65), "does not have 2 blocks")
    raises(lambda: qmm.mx4_dequantize(u8(4, 32), u8(4, 2), 32), "does not have 2 blocks")
    raises(lambda: qmm.mx4_dequantize(u8(4, 32), u8(4, 2), 64), "GPU tensors")
    raises(lambda: qmm.mx4_dequantize(x, u8(4, 2)), "codes must be uint8")
    raises(lambda: qmm.mx4_pack(x, u8(4, 2)), "codes must be a uint8")
    raises(lambda: qmm.mx4_pack(u8(2, 4, 32), u8(4, 2)), "both")
    raises(lambda: qmm.mx4_pack(u8(2, 4, 32), u8(2, 3, 2)), "scales must be")
    raises(lambda: qmm.mx4_pack(u8(4, 32), u8(4, 2)), "GPU tensors")
    raises(lambda: qmm.mx4_gemm(x, W, 32), "GPU tensors")
    raises(lambda: qmm.mx4_gemm(x, W, 48), "must hold")
    raises(lambda: qmm.mx4_gemm(x, W.int(), 32), "W must be a uint8")
    raises(lambda: qmm.mx4_gemm(u8(4, 32), W, 32), "needs its scales")
    raises(lambda: qmm.mx4_gemm(x, W, 32, sx=u8(4, 2)), "goes with uint8")
    raises(lambda: qmm.mx4_gemm(u8(4, 32), W, 32, sx=u8(4, 3)), "scales must be")
    raises(lambda: qmm.mx4_gemm(x[0], W, 32), "2-D")
    raises(lambda: qmm.mx4_gemm(x, W, 32, out=torch.zeros(4, 31)), "GPU tensors")
    up, down = u8(8, qmm.mx4_packed_bytes(32, 64)), u8(8, qmm.mx4_packed_bytes(64, 32))
    lg, ids, w = torch.zeros(4, 8), torch.zeros((4, 2), dtype=torch.int32), torch.zeros(4, 2)
    go = lambda **o: qmm.mx4_moe(*[{**dict(x=x, g=up, u=up, d=down, I=32), **o}[n] for n in "xgudI"],  # noqa: E731
                                 **{k: v for k, v in o.items() if k not in "xgudI"})
    raises(lambda: go(logits=lg, top_k=2), "GPU tensors")
    raises(lambda: go(logits=lg), "need top_k")
    raises(lambda: go(logits=lg, top_k=2, ids=ids), "not both")
    raises(lambda: go(), "must be given")
    raises(lambda: go(ids=ids), "must be given")
    raises(lambda: go(logits=lg[:, :7], top_k=2), "logits must be")
    raises(lambda: go(logits=lg.int(), top_k=2), "logits must be one of")
    raises(lambda: go(ids=ids.short(), weights=w), "int32 or int64")
    raises(lambda: go(ids=ids, weights=w[:, :1].contiguous()), "weights must be")
    raises(lambda: go(ids=ids[:3], weights=w), "ids must be a contiguous (4, k)")
    raises(lambda: go(ids=ids, weights=w, top_k=3), "ids has 2")
    raises(lambda: go(logits=lg, top_k=2, act="relu"), "act must be one of")
    raises(lambda: go(logits=lg, top_k=2, g=up[0]), "Wg must be (E, bytes)")
    raises(lambda: go(logits=lg, top_k=2, I=48), "must hold")
    raises(lambda: go(logits=lg, top_k=2, u=up[:7]), "Wu must hold")
    raises(lambda: go(logits=lg, top_k=2, x=x.double()), "x must be one of")


@pytest.mark.parametrize("v", [1 << 32 | 32, 1 << 31, -1, 32.0, None, "32"])
def test_binding_refuses_sizes_that_would_be_cut_off(v):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    x, W = torch.zeros(4, 64), u8(qmm.mx4_packed_bytes(32, 64))
    up, down = u8(8, qmm.mx4_packed_bytes(32, 64)), u8(8, qmm.mx4_packed_bytes(64, 32))
    raises(lambda: qmm.mx4_gemm(x, W, v), "N must be a size")
    raises(lambda: qmm.mx4_moe(x, up, up, down, v, logits=torch.zeros(4, 8), top_k=2), "I must be a size")
    if v is not None:
        raises(lambda: qmm.mx4_moe(x, up, up, down, 32, logits=torch.zeros(4, 8), top_k=v), "top_k must be a size")
        raises(lambda: qmm.mx4_dequantize(u8(4, 32), u8(4, 2), v), "K must be a size")
    if isinstance(v, int):
        assert qmm.mx4_packed_bytes(v, 64) == qmm.mx4_packed_bytes(64, v) == 0


def test_quantizer_reference_worked_example():
    """Largest 6: floor(log2 6) - 2 = 0, scale byte 127 and codes the values themselves, rounded; halves to even."""
    x = torch.zeros(2, 33)
    x[0, :12] = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.26, -5.1, 7.9, -0.2])
    x[0, 32] = 0.375  # a block of its own: 2^-2 2^-2 times 6
    q, s = m4.quantize_ref(x)
    assert m4.unpack(q)[0, :12].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 9, 15, 7, 8]
    assert s.tolist() == [[127, 123], [0, 0]] and m4.unpack(q)[0, 32] == 7 and not m4.unpack(q)[1].any()
    assert m4.values_ref(q, s, 33)[0, 32] == 0.375


def test_values_reference_by_the_bits():
    for c in range(16):
        e, m = c >> 1 & 3, c & 1
        v = (m / 2 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)) * (-1 if c & 8 else 1)
        assert float(m4.VALUES[c]) == v
    assert m4.scale_ref(torch.tensor([0, 1, 127, 254], dtype=torch.uint8)).tolist() == [2.0 ** -127, 2.0 ** -126, 1.0, 2.0 ** 127]
    assert math.isnan(m4.scale_ref(torch.tensor([255], dtype=torch.uint8)))


def test_route_reference_worked_example():
    lg = torch.tensor([[0.0, math.log(3), -math.inf, math.log(3)], [-math.inf, 1.0, -math.inf, -math.inf]])
    ids, w = m4.route_ref(lg, 3, True)
    assert ids.tolist() == [[1, 3, 0], [1, -1, -1]]
    assert torch.allclose(w, torch.tensor([[3, 3, 1], [7, 0, 0]]).double() / 7, rtol=1e-6)
    assert torch.allclose(m4.route_ref(lg, 1, False)[1], torch.tensor([[3 / 7], [1.0]]).double(), rtol=1e-6)


def test_binding_takes_the_longest_rows():
    """Sizes up to 2^20 - 1: their last block is whole in the codes, 2^20 values."""
    K = (1 << 20) - 1
    codes, scales = torch.zeros((2, 1 << 19), dtype=torch.uint8), torch.zeros((2, 1 << 15), dtype=torch.uint8)
    W = torch.zeros(qmm.mx4_packed_bytes(3, K), dtype=torch.uint8)
    assert W.numel() == 4352 * 2048
    raises(lambda: qmm.mx4_gemm(codes, W, 3, sx=scales), "GPU tensors")
    raises(lambda: qmm.mx4_gemm(torch.zeros(2, K), W, 3), "GPU tensors")
    raises(lambda: qmm.mx4_pack(codes, scales), "GPU tensors")
    raises(lambda: qmm.mx4_dequantize(codes, scales, K), "GPU tensors")
    assert L.qmm_mx4_workspace_bytes(2, K, qmm.QMM_MX4) == 4352 * 2048
