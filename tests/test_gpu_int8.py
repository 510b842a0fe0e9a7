"""int8 x int8 operators on the GPU against 64-bit references: every output
within a bound that counts the roundings (int8_util), at sizes from one token
and one column to several tiles, odd ones, strided operands, every type."""
import math

import pytest
import torch

import int8_util as u8
from int8_util import TYPES, U

qmm = pytest.importorskip("gemv_only_quant_amd")
pytestmark = pytest.mark.gpu

# (M, N, K): single elements, below and across tiles of 16 / 64 / 128 / 256 in each
# axis, K not a multiple of 16, 64 or 256
SIZES = [(1, 1, 1), (1, 17, 33), (1, 300, 1024), (2, 64, 4096), (3, 64, 64), (4, 1000, 2050),
         (5, 100, 257), (8, 96, 528), (15, 48, 3000), (16, 130, 1000), (17, 33, 128), (33, 515, 260),
         (64, 256, 512), (65, 129, 300), (100, 1024, 96), (200, 70, 96), (257, 260, 784),
         (300, 520, 1040), (513, 700, 2064),
         # more 128 x 128 tiles than CUs, then enough 256 x 256 ones, ragged in every axis
         (2100, 2100, 300), (2300, 1900, 145), (4090, 1030, 1024), (2950, 2900, 145), (1500, 2900, 200),
         # the longest rows that a few tokens' codes are kept in LDS for, and longer
         (4, 48, 16384), (1, 40, 65536), (2, 20, 40000), (4, 36, 16400)]


def grad_in(m, n, seed, t):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((m, n), generator=g) * 0.25).to(t)


# ------------------------------------------------------------------ quantizer
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("m,k", [(1, 1), (3, 15), (5, 16), (2, 511), (7, 512), (4, 513), (3, 2048),
                                 (3, 4097), (2, 8192), (2, 14336), (2, 16385), (1, 40000), (70, 130)])
def test_quantize_exact(m, k, t):
    x = u8.tokens(m, k, seed=m * 1000 + k, dtype=TYPES[t])
    q, s = qmm.quantize_tokens(x.cuda())
    rq, rs = u8.quantize_ref(x)
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(q.cpu(), rq)
    # the bytes up to whole 16 are zero
    whole = q.as_strided((m, q.stride(0)), (q.stride(0), 1)).cpu()
    assert not whole[:, k:].any()


def test_quantize_ties_and_neighbours():
    """Quotients at and next to halves: x / s = h exactly (s a power of two), and the
    neighbours of h s on both sides."""
    s = 2.0 ** -5
    h = torch.arange(-126.5, 127.0, 1.0)
    v = torch.cat([h * s, torch.nextafter(h * s, torch.tensor(9.0)),
                   torch.nextafter(h * s, torch.tensor(-9.0)), torch.tensor([127 * s])])
    rows = [v]
    for seed in range(40):  # scales that are no power of two: the nearest x to each half
        g = torch.Generator().manual_seed(seed)
        sc = (torch.rand(1, generator=g) + 0.5) * 2.0 ** float(torch.randint(-20, 20, (1,), generator=g))
        top = (sc * 127).float()
        sc = (top.double() / 127).float()
        x = (h.double() * sc.double()).float()
        rows.append(torch.cat([x, torch.nextafter(x, torch.tensor(math.inf)),
                               torch.nextafter(x, torch.tensor(-math.inf)), top]))
    x = torch.stack(rows)
    q, s = qmm.quantize_tokens(x.cuda())
    rq, rs = u8.quantize_ref(x)
    assert torch.equal(s.cpu(), rs) and torch.equal(q.cpu(), rq)


def test_quantize_extremes():
    """Zero rows, subnormal and largest values, infinities and NaN."""
    k = 100
    x = torch.zeros((9, k))
    x[1, 5] = 1e-45
    x[2] = torch.linspace(-1, 1, k) * 1e-40
    x[3] = torch.linspace(-1, 1, k) * 3e38
    x[4] = torch.linspace(-1, 1, k) * 2e-38
    x[5, 7] = math.inf
    x[6, 9] = math.nan
    x[7, 3], x[7, 4] = -math.inf, math.nan
    x[8] = torch.linspace(-3, 2, k)
    q, s = qmm.quantize_tokens(x.cuda())
    rq, rs = u8.quantize_ref(x)
    assert torch.equal(s.cpu().nan_to_num(nan=-1.0), rs.nan_to_num(nan=-1.0))
    assert torch.equal(q.cpu(), rq)


def test_quantize_strided_and_unaligned():
    base = u8.tokens(20, 700, seed=3, dtype=torch.bfloat16).cuda()
    for x in (base[:, 3:300], base[::2, 16:528], base[5:6, 1:2], base[:, :0]):
        q, s = qmm.quantize_tokens(x)
        rq, rs = u8.quantize_ref(x.cpu())
        assert torch.equal(s.cpu(), rs) and torch.equal(q.cpu(), rq)


# ------------------------------------------------------------------ forward
def left(m, k, seed, kind):
    """The call's left operand (on the GPU) and its codes and scales."""
    if kind == "codes":
        g = torch.Generator().manual_seed(seed)
        q, sx = u8.codes(m, k, g, -128, 127), (0.5 + torch.rand(m, generator=g)) / 60.0
        return dict(x=u8.cuda(q), sx=sx.cuda()), q, sx
    x = u8.tokens(m, k, seed, TYPES[kind])
    return dict(x=x.cuda()), *u8.quantize_ref(x)


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("kind,out", [("codes", "fp32"), ("bf16", "bf16"), ("fp16", "fp16"),
                                      ("fp32", "fp32")])
def test_gemm(m, n, k, kind, out):
    a, q, sx = left(m, k, m + n + k, kind)
    w, sw = u8.weight(n, k, seed=n + 7)
    y = qmm.w8a8_gemm(W=u8.cuda(w), sw=sw.cuda(), out_dtype=TYPES[out], **a)
    assert y.dtype == TYPES[out]
    ref = u8.product_ref(q, sx, w, sw)
    u8.assert_close(y, ref, u8.gemm_bound(ref, TYPES[out]), f"gemm {m} {n} {k}")


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("act,kind,out", [("silu", "codes", "fp32"), ("silu", "bf16", "bf16"),
                                          ("gelu", "fp16", "fp16"), ("gelu_tanh", "fp32", "fp32"),
                                          ("gelu", "codes", "fp32")])
def test_gated(m, n, k, act, kind, out):
    a, q, sx = left(m, k, m + n + k + 1, kind)
    wg, sg = u8.weight(n, k, seed=n + 8)
    wu, su = u8.weight(n, k, seed=n + 9)
    sg = sg * 3.0  # activations over their whole bend
    h = qmm.w8a8_gated(a["x"], u8.cuda(wg), sg.cuda(), u8.cuda(wu), su.cuda(), act=act,
                       sx=a.get("sx"), out_dtype=TYPES[out])
    g, u = u8.product_ref(q, sx, wg, sg), u8.product_ref(q, sx, wu, su)
    ref, _ = u8.gated_ref(act, g, u)
    u8.assert_close(h, ref, u8.gated_bound(act, g, u, TYPES[out]), f"gated {act} {m} {n} {k}")


@pytest.mark.parametrize("m", [1, 3, 20, 130])
def test_long_sums_are_exact(m):
    """Every product 127 * 128 in size: sums up to 2^31, one rounding to fp32."""
    n, k = 18, (1 << 17) - 1
    q = torch.full((m, u8.pad16(k)), 127, dtype=torch.int8)[:, :k]
    w = torch.full((n, u8.pad16(k)), -128, dtype=torch.int8)[:, :k]
    w[1::2] = 127
    one = torch.ones(max(m, n)).cuda()
    y = qmm.w8a8_gemm(u8.cuda(q), u8.cuda(w), one[:n], sx=one[:m]).cpu()
    assert torch.equal(y[:, 0], torch.full((m,), float(-127 * 128 * k)))
    assert torch.equal(y[:, 1], torch.full((m,), float(127 * 127 * k)))


@pytest.mark.parametrize("m", [1, 4, 13, 70, 300])
def test_small_sums_are_exact(m):
    """Unit scales: fp32 outputs equal the whole sums (below 2^24)."""
    n, k = 77, 900
    g = torch.Generator().manual_seed(m)
    q, w = u8.codes(m, k, g, -128, 127), u8.codes(n, k, g, -128, 127)
    one = torch.ones(max(m, n)).cuda()
    y = qmm.w8a8_gemm(u8.cuda(q), u8.cuda(w), one[:n], sx=one[:m]).cpu()
    assert torch.equal(y.double(), q.double() @ w.double().t())


@pytest.mark.parametrize("m", [1, 6, 40, 90])
def test_strided_operands_and_outputs(m):
    """Slices of wider tensors in, a slice of a wider tensor out, aligned and not;
    what lies between the output's rows stays."""
    n, k = 70, 200
    g = torch.Generator().manual_seed(5)
    bx = torch.randint(-128, 128, (m + 1, 320), generator=g, dtype=torch.int8).cuda()
    bw = torch.randint(-128, 128, (2 * n, 416), generator=g, dtype=torch.int8).cuda()
    x, w = bx[1:, 16:16 + k], bw[::2, 32:32 + k]
    sx, sw = torch.rand(m, generator=g).cuda(), torch.rand(n, generator=g).cuda()
    ref = u8.product_ref(x.cpu(), sx.cpu(), w.cpu(), sw.cpu())
    for t, at in ((torch.float32, 0), (torch.float32, 1), (torch.bfloat16, 8), (torch.float16, 3)):
        big = torch.full((m, n + 33), 7.0, dtype=t, device="cuda")
        out = big[:, at:at + n]
        assert qmm.w8a8_gemm(x, w, sw, sx=sx, out=out) is out
        u8.assert_close(out, ref, u8.gemm_bound(ref, t), f"strided {t} {at}")
        keep = torch.ones(n + 33, dtype=torch.bool)
        keep[at:at + n] = False
        assert (big.cpu()[:, keep] == 7.0).all()


@pytest.mark.parametrize("m", [1, 3, 30, 100])
def test_padding_takes_no_part(m):
    """K % 16 != 0: bytes past a row's end change nothing."""
    n, k = 40, 145
    g = torch.Generator().manual_seed(11)
    q, w = u8.codes(m, k, g), u8.codes(n, k, g)
    s = torch.rand(max(m, n), generator=g).cuda()
    got = []
    for fill in (0, 127, -128):
        qq, ww = u8.cuda(q), u8.cuda(w)
        qq.as_strided((m, 160), (160, 1))[:, k:] = fill
        ww.as_strided((n, 160), (160, 1))[:, k:] = -1 - fill
        y = qmm.w8a8_gemm(qq, ww, s[:n], sx=s[:m])
        d = grad_in(m, n, 4, torch.bfloat16).cuda()
        got.append([y, *qmm.w8a8_gemm_backward(d, qq, s[:m], ww, s[:n]),
                    *qmm.w8a8_gated_backward(d, qq, s[:m], ww, s[:n], ww, s[:n])])
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a, b)


def test_rows_that_are_not_finite_touch_no_other():
    for m in (2, 30, 130):
        n, k = 50, 300
        x = u8.tokens(m, k, seed=1)
        x[m // 2, 7] = math.inf
        x[0] = 0.0
        w, sw = u8.weight(n, k, seed=2)
        y = qmm.w8a8_gemm(x.cuda(), u8.cuda(w), sw.cuda()).cpu()
        h = qmm.w8a8_gated(x.cuda(), u8.cuda(w), sw.cuda(), u8.cuda(w), sw.cuda()).cpu()
        for o in (y, h):
            assert torch.isnan(o[m // 2]).all()
            o[m // 2] = 0
            assert torch.isfinite(o).all() and (o[0] == 0).all()


@pytest.mark.parametrize("act", qmm.ACTIVATIONS)
def test_activation_at_its_ends(act):
    """Gates from -1e30 to 1e30: h stays the limit (0 or g u), never NaN; NaN stays NaN."""
    for m in (1, 40, 80):
        n, k = 12, 16
        q = torch.zeros((m, k), dtype=torch.int8)
        q[:, 0] = 1
        w = torch.zeros((n, k), dtype=torch.int8)
        w[:, 0] = 1
        sg = torch.tensor([0.0, 1e-30, -1e-3, 1.0, -1.0, 30.0, -30.0, -90.0, 200.0, 1e30, -1e30, math.nan])
        su = torch.full((n,), 2.0)
        h = qmm.w8a8_gated(q.cuda(), w.cuda(), sg.cuda(), w.cuda(), su.cuda(), act=act,
                           sx=torch.ones(m).cuda()).cpu().double()
        g = sg.double().expand(m, n)
        u = torch.full((m, n), 2.0, dtype=torch.float64)
        ref, amp = u8.gated_ref(act, g, u)
        ref[:, 10] = 0.0
        assert torch.isnan(h[:, 11]).all()
        bound = ref.abs() * (40 + 16 * amp.clamp(max=1e6)) * U + 2.0 ** -120
        bound[:, 9] = 1e30 * 8 * U
        u8.assert_close(h[:, :11], ref[:, :11], bound[:, :11], f"ends {act} {m}")


# ------------------------------------------------------------------ gradients
GRAD_SIZES = [(1, 1, 1), (1, 64, 33), (3, 17, 64), (16, 130, 200), (64, 128, 256), (65, 129, 300),
              (130, 300, 70), (257, 260, 500), (300, 520, 1040), (129, 700, 2064),
              # many rows (dx, and the gated block's g and u); contractions long enough to be
              # split over workgroups (dW in the first and last, dx in the second)
              (2100, 70, 2100), (70, 2100, 130), (1000, 2060, 90), (4200, 40, 60), (2950, 40, 2900),
              (1500, 2900, 90)]


@pytest.mark.parametrize("m,n,k", GRAD_SIZES)
@pytest.mark.parametrize("t", ["bf16", "fp16"])
def test_gemm_backward(m, n, k, t):
    t = TYPES[t]
    q, sx = u8.quantize_ref(u8.tokens(m, k, seed=k))
    w, sw = u8.weight(n, k, seed=n)
    dy = grad_in(m, n, m, t)
    qc = u8.codes(m, k, torch.Generator().manual_seed(0))  # padded rows
    qc.copy_(q)
    dx, dw = qmm.w8a8_gemm_backward(dy.cuda(), u8.cuda(qc), sx.cuda(), u8.cuda(w), sw.cuda())
    rx, rw = u8.backward_ref(dy, q, sx, w, sw)
    bx, bw = u8.backward_bound(dy, q, sx, w, sw, t)
    assert dx.dtype == dw.dtype == t
    u8.assert_close(dx, rx, bx, "dx")
    u8.assert_close(dw, rw, bw, "dW")
    alone, none = qmm.w8a8_gemm_backward(dy.cuda(), None, None, u8.cuda(w), sw.cuda(), weight_grad=False)
    assert none is None and torch.equal(alone, dx)


@pytest.mark.parametrize("m,n,k", GRAD_SIZES)
@pytest.mark.parametrize("act,t", [("silu", "bf16"), ("gelu", "fp16"), ("gelu_tanh", "bf16")])
def test_gated_backward(m, n, k, act, t):
    t = TYPES[t]
    q, sx = u8.quantize_ref(u8.tokens(m, k, seed=k + 1))
    qc = u8.codes(m, k, torch.Generator().manual_seed(0))
    qc.copy_(q)
    wg, sg = u8.weight(n, k, seed=n + 1)
    wu, su = u8.weight(n, k, seed=n + 2)
    sg = sg * 2.0
    dh = grad_in(m, n, m + 1, t)
    args = (u8.cuda(qc), sx.cuda(), u8.cuda(wg), sg.cuda(), u8.cuda(wu), su.cuda())
    got = qmm.w8a8_gated_backward(dh.cuda(), *args, act=act)
    refs = u8.gated_backward_ref(act, dh, q, sx, wg, sg, wu, su)
    bounds = u8.gated_backward_bound(act, dh, q, sx, wg, sg, wu, su, t)
    for name, o, r, b in zip(("dx", "dWg", "dWu"), got, refs, bounds):
        assert o.dtype == t
        u8.assert_close(o, r, b, name)
    alone, a, b = qmm.w8a8_gated_backward(dh.cuda(), *args, act=act, weight_grad=False)
    assert a is None and b is None and torch.equal(alone, got[0])


def _along(f, v, eps=1e-4):
    return (f(eps * v) - f(-eps * v)).double().sum() / (2 * eps)


@pytest.mark.parametrize("act", qmm.ACTIVATIONS)
def test_gated_backward_against_differences(act):
    """Along random directions, sum(grad * v) against central differences of the
    forward formula in 64 bits; off by at most the outputs' bounds along |v| and by
    the differences' own eps^2 (1e-8 of the terms' size, taken 100 times)."""
    m, n, k, t = 40, 60, 90, torch.bfloat16
    q, sx = u8.quantize_ref(u8.tokens(m, k, seed=1))
    qc = u8.codes(m, k, torch.Generator().manual_seed(0))
    qc.copy_(q)
    wg, sg = u8.weight(n, k, seed=2)
    wu, su = u8.weight(n, k, seed=3)
    dh = grad_in(m, n, 4, t)
    got = qmm.w8a8_gated_backward(dh.cuda(), u8.cuda(qc), sx.cuda(), u8.cuda(wg), sg.cuda(),
                                  u8.cuda(wu), su.cuda(), act=act)
    bounds = u8.gated_backward_bound(act, dh, q, sx, wg, sg, wu, su, t)
    xh = q.double() * sx.double()[:, None]
    gh, uh = wg.double() * sg.double()[:, None], wu.double() * su.double()[:, None]

    def loss(dx=0.0, dg=0.0, du=0.0):
        g, u = (xh + dx) @ (gh + dg).t(), (xh + dx) @ (uh + du).t()
        return u8.act_ref(act, g)[0] * u * dh.double()

    for name, o, b in zip(("dx", "dg", "du"), got, bounds):
        for seed in range(3):
            v = torch.randn(o.shape, generator=torch.Generator().manual_seed(seed)).double()
            want = _along(lambda s: loss(**{name: s}), v)
            have = (o.double().cpu() * v).sum()
            assert (want - have).abs() <= (b * v.abs()).sum() + 1e-6 * (o.double().cpu() * v).abs().sum()


def test_gemm_backward_against_differences():
    m, n, k, t = 30, 50, 70, torch.float16
    q, sx = u8.quantize_ref(u8.tokens(m, k, seed=1))
    qc = u8.codes(m, k, torch.Generator().manual_seed(0))
    qc.copy_(q)
    w, sw = u8.weight(n, k, seed=2)
    dy = grad_in(m, n, 4, t)
    got = qmm.w8a8_gemm_backward(dy.cuda(), u8.cuda(qc), sx.cuda(), u8.cuda(w), sw.cuda())
    bounds = u8.backward_bound(dy, q, sx, w, sw, t)
    xh, wh = q.double() * sx.double()[:, None], w.double() * sw.double()[:, None]
    fs = (lambda s: (xh + s) @ wh.t() * dy.double(), lambda s: xh @ (wh + s).t() * dy.double())
    for f, o, b in zip(fs, got, bounds):
        v = torch.randn(o.shape, generator=torch.Generator().manual_seed(9)).double()
        have = (o.double().cpu() * v).sum()
        assert (_along(f, v) - have).abs() <= (b * v.abs()).sum() + 1e-6 * (o.double().cpu() * v).abs().sum()


# whole rounds of 256 x 256 tiles: of g and u made again; of dx (the contraction over
# both weights); of dW (the rows of both)
@pytest.mark.parametrize("m,n,k,t", [(4000, 2000, 1000, "bf16"), (4000, 650, 4090, "fp16"),
                                     (1300, 2000, 4090, "bf16")])
def test_gated_backward_in_the_largest_tiles(m, n, k, t):
    test_gated_backward(m, n, k, "silu", t)


@pytest.mark.parametrize("m,n,k,t", [(4000, 1300, 4090, "bf16"), (1300, 4000, 4090, "fp16")])
def test_gemm_backward_in_the_largest_tiles(m, n, k, t):
    test_gemm_backward(m, n, k, t)


def test_forward_in_the_largest_tiles():
    test_gemm(4090, 4000, 1000, "codes", "bf16")
    test_gated(4090, 2000, 1000, "silu", "codes", "fp32")


@pytest.mark.parametrize("m", [3, 70, 300])
def test_gradients_that_are_not_finite_stay_in_their_rows(m):
    """An infinity in one incoming gradient reaches that token's dx and that
    column's dW, and nothing else."""
    n, k, t = 90, 130, torch.bfloat16
    q, sx = u8.quantize_ref(u8.tokens(m, k, seed=1))
    wg, sg = u8.weight(n, k, seed=2)
    wu, su = u8.weight(n, k, seed=3)
    qc = u8.codes(m, k, torch.Generator().manual_seed(0))
    qc.copy_(q)
    dy = grad_in(m, n, 4, t)
    dy[m // 2, 7] = math.inf
    args = (u8.cuda(qc), sx.cuda(), u8.cuda(wg), sg.cuda())
    dx, dw = qmm.w8a8_gemm_backward(dy.cuda(), *args)
    gx, gw, uw = qmm.w8a8_gated_backward(dy.cuda(), *args, u8.cuda(wu), su.cuda())
    for o, bad in ((dx, m // 2), (gx, m // 2), (dw, 7), (gw, 7), (uw, 7)):
        fine = torch.isfinite(o).all(1)
        assert not fine[bad] and int(fine.sum()) == o.shape[0] - 1


@pytest.mark.parametrize("m", [1, 65])
def test_infinite_scale_stays_in_its_column(m):
    """An up projection's infinite scale: du of that column is finite, and so is dWu;
    dWg of it is infinite with the sign of its sum (every term has it), not NaN for the
    tokens that only pad a tile."""
    n, k, t = 20, 16, torch.bfloat16
    q = torch.full((m, k), 5, dtype=torch.int8)
    sx = torch.full((m,), 0.125)
    wg = torch.ones((n, k), dtype=torch.int8)
    sw = torch.full((n,), 0.25)
    su = sw.clone()
    su[7] = math.inf
    dh = torch.full((m, n), 0.5, dtype=t)
    dx, gw, uw = qmm.w8a8_gated_backward(dh.cuda(), q.cuda(), sx.cuda(), wg.cuda(), sw.cuda(), wg.cuda(),
                                         su.cuda())
    assert torch.isfinite(uw).all() and not torch.isfinite(dx).any()
    fine = torch.isfinite(gw).all(1)
    assert int(fine.sum()) == n - 1 and (gw[7] == math.inf).all()


def test_backward_small_scales_in_fp16():
    """Scales of 1e-7: dy sw would be subnormal in fp16 without the power of two."""
    m, n, k, t = 40, 64, 64, torch.float16
    q, sx = u8.quantize_ref(u8.tokens(m, k, seed=1) * 1e-6)
    w, _ = u8.weight(n, k, seed=2)
    sw = torch.full((n,), 3e-3)
    dy = grad_in(m, n, 4, t)
    dx, dw = qmm.w8a8_gemm_backward(dy.cuda(), q.cuda(), sx.cuda(), w.cuda(), sw.cuda())
    rx, rw = u8.backward_ref(dy, q, sx, w, sw)
    bx, bw = u8.backward_bound(dy, q, sx, w, sw, t)
    u8.assert_close(dx, rx, bx, "dx")
    u8.assert_close(dw, rw, bw, "dW")


def test_strided_gradients():
    m, n, k = 37, 45, 80
    base = grad_in(m, 3 * n, 1, torch.bfloat16)
    q, sx = u8.quantize_ref(u8.tokens(m, k, seed=1))
    w, sw = u8.weight(n, k, seed=2)
    for at in (0, 1, 16):
        dy = base[:, at:at + n]
        dx, dw = qmm.w8a8_gemm_backward(base.cuda()[:, at:at + n], q.cuda(), sx.cuda(), w.cuda(), sw.cuda())
        rx, rw = u8.backward_ref(dy, q, sx, w, sw)
        bx, bw = u8.backward_bound(dy, q, sx, w, sw, torch.bfloat16)
        u8.assert_close(dx, rx, bx, "dx")
        u8.assert_close(dw, rw, bw, "dW")


# ------------------------------------------------------------------ empty sums, streams, graphs
def test_empty_sums_are_zero():
    z = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    i8 = torch.int8
    f = torch.float32
    assert (qmm.w8a8_gemm(z(3, 0), z(5, 0, t=i8), z(5, t=f).fill_(1)) == 0).all()
    assert (qmm.w8a8_gated(z(3, 0), z(5, 0, t=i8), z(5, t=f), z(5, 0, t=i8), z(5, t=f)) == 0).all()
    assert qmm.w8a8_gemm(z(0, 16), z(5, 16, t=i8), z(5, t=f)).shape == (0, 5)
    assert qmm.w8a8_gemm(z(4, 16), z(0, 16, t=i8), z(0, t=f)).shape == (4, 0)
    dx, dw = qmm.w8a8_gemm_backward(z(0, 5), z(0, 16, t=i8), z(0, t=f), z(5, 16, t=i8), z(5, t=f))
    assert dx.shape == (0, 16) and (dw == 0).all()
    dx, dw = qmm.w8a8_gemm_backward(z(4, 0), z(4, 16, t=i8), z(4, t=f), z(0, 16, t=i8), z(0, t=f))
    assert (dx == 0).all() and dw.shape == (0, 16)
    dx, a, b = qmm.w8a8_gated_backward(z(0, 5), z(0, 16, t=i8), z(0, t=f), z(5, 16, t=i8), z(5, t=f),
                                       z(5, 16, t=i8), z(5, t=f))
    assert (a == 0).all() and (b == 0).all()
    q, s = qmm.quantize_tokens(z(3, 0))
    assert q.shape == (3, 0) and (s == 0).all()


def _calls(m):
    n, k = 330, 500
    w, sw = u8.weight(n, k, seed=1)
    v, sv = u8.weight(n, k, seed=2)
    x = u8.tokens(m, k, seed=3, dtype=torch.bfloat16).cuda()
    d = grad_in(m, n, 4, torch.bfloat16).cuda()
    w, sw, v, sv = u8.cuda(w), sw.cuda(), u8.cuda(v), sv.cuda()

    def step():
        q, s = qmm.quantize_tokens(x)
        return [qmm.w8a8_gemm(x, w, sw), qmm.w8a8_gated(q, w, sw, v, sv, sx=s),
                *qmm.w8a8_gemm_backward(d, q, s, w, sw), *qmm.w8a8_gated_backward(d, q, s, w, sw, v, sv)]
    return step, x


@pytest.mark.parametrize("m", [1, 20, 150])
def test_graph_replays_equal_eager(m):
    step, x = _calls(m)
    other, _ = _calls(m + 3)
    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(3):
        for o in outs:
            o.fill_(7)
        other()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for o, r in zip(outs, want):
            assert torch.equal(o, r)


@pytest.mark.parametrize("m", [1, 20, 150])
def test_other_stream_and_repeat(m):
    """The current stream is the one used; a repeat gives the same bits."""
    step, _ = _calls(m)
    want = [t.clone() for t in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ together
def _example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "int8_feed_forward.py")
    spec = importlib.util.spec_from_file_location("int8_feed_forward", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_layer_is_the_same_for_one_token_and_many():
    """The sums are whole numbers and every kernel rounds the same steps, so a
    token's output does not depend on what is computed beside it."""
    layer = _example().FeedForward(512, 700)
    x = u8.tokens(600, 512, seed=5, dtype=torch.bfloat16).cuda()
    whole = layer.serve(x)
    for a, b in ((0, 1), (3, 6), (10, 30), (40, 100), (100, 400)):
        assert torch.equal(layer.serve(x[a:b]), whole[a:b]), (a, b)


def test_layer_trains():
    losses = _example().train(tokens=256, width=256, hidden=704, steps=12, rate=0.3, log=lambda *_: None)
    assert all(math.isfinite(v) for v in losses)
    assert losses[-1] < 0.7 * losses[0], losses
