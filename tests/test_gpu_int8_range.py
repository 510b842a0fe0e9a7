"""fp16 gradients of the int8 x int8 operators over fp16's whole range, against
64-bit references: products that leave the range although the results do not,
and rows of very different size beside each other.

Each row of a gradient's product has a power of two of its own, so that its small
values lose what they lose of the row's largest value, whatever other rows hold.
The bounds here count, for an operand d, half a step of d and 2^-30 of its row's
largest (the row's largest value is kept at 2^7 or more, a step among subnormals
is 2^-24, and a value may be rounded there twice: 2 * 2^-25 / 2^7 = 2^-31), the
sum's fp32 roundings, and the result's own."""
import pytest
import torch

import int8_util as u8
from int8_util import U

qmm = pytest.importorskip("gemv_only_quant_amd")
pytestmark = pytest.mark.gpu
F16 = torch.float16


def row_bound(d, derr, codes_):
    """|sum d c| with d an operand in fp16 (rows are output rows)."""
    step = u8.half(F16) + (d.shape[1] + 4) * U
    return (d.abs() * step + derr + 2.0 ** -30 * d.abs().amax(1, keepdim=True)) @ codes_.double().abs()


def operands(m, n, k, xsize, wsize, seed):
    """Codes and scales of rows of size xsize, and two weights whose rows have the
    scale wsize / 127, up to 10%."""
    q, sx = u8.quantize_ref(u8.tokens(m, k, seed) * xsize)
    qc = u8.codes(m, k, torch.Generator().manual_seed(0))
    qc.copy_(q)
    ws = []
    for i in (1, 2):
        g = torch.Generator().manual_seed(seed + i)
        ws += [u8.codes(n, k, g), (0.9 + 0.1 * torch.rand(n, generator=g)) * (wsize / 127)]
    return qc, sx, ws


def linear_refs(dy, q, sx, w, sw):
    refs = u8.backward_ref(dy, q, sx, w, sw)
    d = dy.double() * sw.double()
    t = (dy.double() * sx.double()[:, None]).t()
    return refs, [row_bound(d, torch.zeros_like(d), w) + u8.round_bound(refs[0], F16),
                  row_bound(t, torch.zeros_like(t), q) + u8.round_bound(refs[1], F16)]


@pytest.mark.parametrize("m,n,k", [(512, 300, 200), (40, 130, 70), (1100, 64, 300)])
@pytest.mark.parametrize("size,spread", [(1e-3, 1e4), (1e-4, 1e3), (0.25, 1e5)])
def test_dw_beside_one_loud_token(m, n, k, size, spread):
    """One token's scale is `spread` times the others', and its gradient zero."""
    q, sx, (w, sw, _, _) = operands(m, n, k, 1.0, 1.0, seed=1)
    sx[m // 3] *= spread
    dy = (torch.randn((m, n), generator=torch.Generator().manual_seed(2)) * size).to(F16)
    dy[m // 3] = 0
    dx, dw = qmm.w8a8_gemm_backward(dy.cuda(), u8.cuda(q), sx.cuda(), u8.cuda(w), sw.cuda())
    for got, ref, b, what in zip((dx, dw), *linear_refs(dy, q, sx, w, sw), ("dx", "dW")):
        u8.assert_close(got, ref, b, what)


@pytest.mark.parametrize("m,n,k", [(512, 300, 200), (5, 1100, 70), (300, 64, 300)])
@pytest.mark.parametrize("size,spread", [(1e-3, 1e4), (1e-4, 1e3), (0.25, 1e5)])
def test_dx_beside_one_loud_channel(m, n, k, size, spread):
    """One output channel's scale is `spread` times the others', and its gradient zero."""
    q, sx, (w, sw, _, _) = operands(m, n, k, 1.0, 1.0, seed=1)
    sw[n // 3] *= spread
    dy = (torch.randn((m, n), generator=torch.Generator().manual_seed(2)) * size).to(F16)
    dy[:, n // 3] = 0
    dx, dw = qmm.w8a8_gemm_backward(dy.cuda(), u8.cuda(q), sx.cuda(), u8.cuda(w), sw.cuda())
    for got, ref, b, what in zip((dx, dw), *linear_refs(dy, q, sx, w, sw), ("dx", "dW")):
        u8.assert_close(got, ref, b, what)
