"""The int8 x int8 operators pass no gradients on by themselves, and say so."""
import warnings

import pytest
import torch

import int8_util as u8

qmm = pytest.importorskip("gemv_only_quant_amd")
pytestmark = pytest.mark.gpu


def _operands():
    w, sw = u8.weight(48, 64, seed=1)
    return torch.randn((8, 64), device="cuda", dtype=torch.float16), w.cuda(), sw.cuda()


def test_a_call_that_drops_gradients_warns():
    x, w, sw = _operands()
    leaf = x.clone().requires_grad_()
    scale = sw.clone().requires_grad_()
    for call in (lambda: qmm.w8a8_gemm(leaf, w, sw), lambda: qmm.w8a8_gemm(x, w, scale),
                 lambda: qmm.w8a8_gated(leaf, w, sw, w, sw), lambda: qmm.quantize_tokens(leaf)):
        with pytest.warns(UserWarning, match="gradients"):
            y = call()
        assert not (y[0] if isinstance(y, tuple) else y).requires_grad


class Linear(torch.autograd.Function):
    """As a user's program would wrap the calls."""

    @staticmethod
    def forward(ctx, x, w, sw):
        xq, sx = qmm.quantize_tokens(x)
        ctx.save_for_backward(xq, sx, w, sw)
        return qmm.w8a8_gemm(xq, w, sw, sx=sx, out_dtype=x.dtype)

    @staticmethod
    def backward(ctx, dy):
        return qmm.w8a8_gemm_backward(dy, *ctx.saved_tensors, weight_grad=False)[0], None, None


def test_no_warning_where_none_are_lost():
    x, w, sw = _operands()
    leaf = x.clone().requires_grad_()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        qmm.w8a8_gemm(x, w, sw)
        with torch.no_grad():
            plain = qmm.w8a8_gemm(leaf, w, sw, out_dtype=x.dtype)
        y = Linear.apply(leaf, w, sw)
        dy = torch.ones_like(y)
        y.backward(dy)
    assert torch.equal(y, plain)
    assert torch.equal(leaf.grad, qmm.w8a8_gemm_backward(dy, None, None, w, sw, weight_grad=False)[0])
