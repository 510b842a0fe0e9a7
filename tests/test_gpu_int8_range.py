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


def sized_grad(shape, lines, act, args, which):
    """An incoming gradient on some of its lines, of the size that brings the largest of
    the results `which` to 30000."""
    dh = torch.zeros(shape, dtype=F16)
    part = dh[lines]
    part.copy_(torch.randn(part.shape, generator=torch.Generator().manual_seed(3)) * 1000)
    top = max(float(u8.gated_backward_ref(act, dh, *args)[i].abs().max()) for i in which)
    return (dh.double() * (30000.0 / top)).to(F16)


def gated_refs(act, dh, q, sx, wg, sg, wu, su):
    """(reference, bound) of dx, dWg and dWu."""
    dg, du, eg, eu = u8.gated_grads(act, dh, q, sx, wg, sg, wu, su)
    # beyond |g| = 30 act' is 0 or 1 and act 0 or g within 2^-36: what is left are u's or
    # g's four roundings, the products' two and the evaluation's few
    g, u = u8.product_ref(q, sx, wg, sg), u8.product_ref(q, sx, wu, su)
    far, d = g.abs() > 30, dh.double()
    eg = torch.where(far, (d * u).abs() * 16 * U, eg)
    eu = torch.where(far, du.abs() * 16 * U + d.abs() * 2.0 ** -30, eu)
    refs = u8.gated_backward_ref(act, dh, q, sx, wg, sg, wu, su)
    s = sx.double()[:, None]
    d, e = (torch.cat([a * sg.double(), b * su.double()], 1) for a, b in ((dg, du), (eg, eu)))
    bounds = [row_bound(d, e, torch.cat([wg, wu], 0)), row_bound((dg * s).t(), (eg * s).t(), q),
              row_bound((du * s).t(), (eu * s).t(), q)]
    return [(r, b + u8.round_bound(r, F16)) for r, b in zip(refs, bounds)], dg, du


def linear_refs(dy, q, sx, w, sw):
    refs = u8.backward_ref(dy, q, sx, w, sw)
    d = dy.double() * sw.double()
    t = (dy.double() * sx.double()[:, None]).t()
    return refs, [row_bound(d, torch.zeros_like(d), w) + u8.round_bound(refs[0], F16),
                  row_bound(t, torch.zeros_like(t), q) + u8.round_bound(refs[1], F16)]


# rows below, of and above a tile; few columns and contractions split over workgroups
SIZES = [(3, 600, 130), (70, 333, 500), (300, 2100, 90), (64, 70, 2100)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("act", qmm.ACTIVATIONS)
def test_gated_dx_where_dg_leaves_the_range(m, n, k, act):
    """Loud activations: dg and du pass 65504, dx does not."""
    q, sx, w = operands(m, n, k, 400.0, 0.03, seed=m)
    dh = sized_grad((m, n), (slice(None), slice(None, None, n // 5)), act, (q, sx, *w), (0,))
    refs, dg, du = gated_refs(act, dh, q, sx, *w)
    assert min(dg.abs().max(), du.abs().max()) > 1e5 and refs[0][0].abs().max() < 65504
    args = [u8.cuda(q), sx.cuda(), *(u8.cuda(t) for t in w)]
    for wgrad in (False, True):
        dx = qmm.w8a8_gated_backward(dh.cuda(), *args, act=act, weight_grad=wgrad)[0]
        u8.assert_close(dx, *refs[0], f"dx, weight_grad={wgrad}")


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("act", qmm.ACTIVATIONS)
def test_gated_dw_where_dg_leaves_the_range(m, n, k, act):
    """Loud weights: dg and du pass 65504, dWg and dWu do not."""
    q, sx, w = operands(m, n, k, 0.01, 600.0, seed=m)
    dh = sized_grad((m, n), slice(None, None, -(-m // 5)), act, (q, sx, *w), (1, 2))
    refs, dg, du = gated_refs(act, dh, q, sx, *w)
    assert min(dg.abs().max(), du.abs().max()) > 1e5
    assert max(refs[1][0].abs().max(), refs[2][0].abs().max()) < 65504
    got = qmm.w8a8_gated_backward(dh.cuda(), u8.cuda(q), sx.cuda(), *(u8.cuda(t) for t in w), act=act)
    u8.assert_close(got[1], *refs[1], "dWg")
    u8.assert_close(got[2], *refs[2], "dWu")


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


# (the last: 256 x 256 tiles where g and u are made again)
@pytest.mark.parametrize("m,n,k", SIZES + [(4000, 2000, 200)])
def test_gated_beside_loud_tokens_and_channels(m, n, k):
    """Token and channel scales over four decades, gradients that undo them in part:
    every row's operands have a size of their own."""
    q, sx, (wg, sg, wu, su) = operands(m, n, k, 1.0, 0.3, seed=2)
    g = torch.Generator().manual_seed(9)
    sx = sx * 10.0 ** (4 * torch.rand(m, generator=g) - 3)
    sg, su = (s * 10.0 ** (2 * torch.rand(n, generator=g) - 1) for s in (sg, su))
    dh = (torch.randn((m, n), generator=g) * 0.05 / (sx[:, None] * 100).clamp(min=0.1)).to(F16)
    refs, _, _ = gated_refs("silu", dh, q, sx, wg, sg, wu, su)
    got = qmm.w8a8_gated_backward(dh.cuda(), u8.cuda(q), sx.cuda(), u8.cuda(wg), sg.cuda(), u8.cuda(wu), su.cuda())
    for o, r, what in zip(got, refs, ("dx", "dWg", "dWu")):
        u8.assert_close(o, *r, what)


@pytest.mark.parametrize("m", [3, 70, 300])
def test_infinite_gradients_stay_in_their_rows_in_fp16(m):
    """An infinity in one incoming gradient reaches that token's dx and that column's dW,
    and leaves the other rows their accuracy."""
    n, k = 90, 130
    q, sx, w = operands(m, n, k, 1.0, 1.0, seed=4)
    dy = (torch.randn((m, n), generator=torch.Generator().manual_seed(2)) * 1e-3).to(F16)
    dy[m // 2, 7] = torch.inf
    args = (u8.cuda(q), sx.cuda())
    dev = [u8.cuda(t) for t in w]
    fine = dy.clone()
    fine[m // 2, 7] = 0
    lin = linear_refs(fine, q, sx, *w[:2])
    gat, _, _ = gated_refs("silu", fine, q, sx, *w)
    outs = list(zip(qmm.w8a8_gemm_backward(dy.cuda(), *args, *dev[:2]), zip(*lin), (m // 2, 7)))
    outs += list(zip(qmm.w8a8_gated_backward(dy.cuda(), *args, *dev), gat, (m // 2, 7, 7)))
    for o, (ref, bound), bad in outs:
        keep = torch.arange(o.shape[0]) != bad
        assert not torch.isfinite(o[bad]).any()
        u8.assert_close(o[keep.cuda()], ref[keep], bound[keep], "other rows")
