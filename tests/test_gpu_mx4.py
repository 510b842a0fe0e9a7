"""Microscaled 4-bit operators on the GPU against 64-bit references: codes, scales and
values exact, sums within bounds that count the roundings (mx4_util)."""
import math

import pytest
import torch

import mx4_util as m4
from mx4_util import TYPES

qmm = pytest.importorskip("gemv_only_quant_amd")
pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ quantizer
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("m,k", [(1, 1), (3, 31), (5, 32), (2, 33), (7, 100), (4, 512), (3, 1000), (64, 2048),
                                 (2, 4097), (1, 14336), (300, 40)])
def test_quantize_exact(m, k, t):
    x = m4.tokens(m, k, seed=m * 1000 + k, dtype=TYPES[t])
    q, s = qmm.mx4_quantize(x.cuda())
    rq, rs = m4.quantize_ref(x)
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(q.cpu(), rq)
    whole = s.as_strided((m, s.stride(0)), (s.stride(0), 1)).cpu()
    assert not whole[:, rs.shape[1]:].any()


@pytest.mark.parametrize("t", TYPES)
def test_quantize_every_border(t):
    """Every border between codes and its neighbours on both sides, at scales from the smallest to the largest."""
    rows = []
    for e in (-149, -140, -130, -127, -126, -125, -120, -30, -17, -14, -3, 0, 1, 9, 13, 60, 124, 125):
        h = torch.tensor([0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 7.75], dtype=torch.float64)
        v = (h * 2.0 ** e).float().to(TYPES[t])
        if not torch.isfinite(v).all():
            continue
        for d in (0, 1, -1):  # neighbours by the bits
            b = (v.view(torch.int32 if t == "fp32" else torch.int16) + d).clamp(min=0)
            rows.append(torch.cat([b.view(v.dtype), -b.view(v.dtype)]))
    x = torch.stack(rows)
    # a block's largest value sets its scale: 4, 5, 6 and 7.75 of them in turn
    x = torch.cat([x, *(torch.where(x.abs() > c * (x.abs().amax(1, keepdim=True) / 7.75), torch.zeros_like(x), x)
                        for c in (6.0, 5.0, 4.0))])
    x = x[torch.isfinite(x.float()).all(1)]
    q, s = qmm.mx4_quantize(x.cuda())
    rq, rs = m4.quantize_ref(x)
    assert torch.equal(s.cpu(), rs) and torch.equal(q.cpu(), rq)


def test_quantize_every_half_value():
    """Every finite 16-bit value, 31 blocks' largest."""
    for t in (torch.float16, torch.bfloat16):
        v = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(t)
        v = v[torch.isfinite(v)]
        x = v[:v.numel() // 32 * 32].reshape(-1, 32)
        x = torch.cat([x, x.flatten()[torch.randperm(x.numel(), generator=torch.Generator().manual_seed(1))].reshape(-1, 32)])
        q, s = qmm.mx4_quantize(x.cuda())
        rq, rs = m4.quantize_ref(x)
        assert torch.equal(s.cpu(), rs) and torch.equal(q.cpu(), rq)


@pytest.mark.parametrize("t", TYPES)
def test_quantize_not_finite_and_zero(t):
    x = m4.tokens(6, 96, seed=1, dtype=TYPES[t])
    x[0] = 0.0
    x[1, 40], x[2, 33], x[3, 95] = math.inf, math.nan, -math.inf
    x[4, :32], x[5, 5] = -0.0, 0.0
    q, s = qmm.mx4_quantize(x.cuda())
    rq, rs = m4.quantize_ref(x)
    assert torch.equal(s.cpu(), rs) and torch.equal(q.cpu(), rq)
    assert rs[1].tolist()[1] == rs[2].tolist()[1] == rs[3].tolist()[2] == 255
    y = qmm.mx4_dequantize(q, s).cpu()
    assert torch.isnan(y[1, 32:64]).all() and torch.isfinite(y[1, :32]).all() and torch.isfinite(y[1, 64:]).all()


def test_quantize_strided_and_unaligned():
    for t in TYPES.values():
        base = m4.tokens(20, 700, seed=3, dtype=t).cuda()
        for x in (base[:, 3:300], base[::2, 16:528], base[5:6, 1:2], base[:, :0], base[:0]):
            q, s = qmm.mx4_quantize(x)
            rq, rs = m4.quantize_ref(x.cpu())
            assert torch.equal(s.cpu(), rs) and torch.equal(q.cpu(), rq)


@pytest.mark.parametrize("t", TYPES)
def test_dequantize_every_code_and_scale(t):
    c = m4.pack(torch.arange(16, dtype=torch.uint8).repeat(2)).expand(256, 16).contiguous()
    s = torch.arange(256, dtype=torch.int32).to(torch.uint8)[:, None]
    y = qmm.mx4_dequantize(c.cuda(), s.cuda(), out_dtype=TYPES[t])
    want = m4.values_ref(c, s).to(TYPES[t])
    assert torch.equal(y.cpu().view(torch.int32 if t == "fp32" else torch.int16)[:255],
                       want.view(torch.int32 if t == "fp32" else torch.int16)[:255])
    assert torch.isnan(y[255]).all()


def test_dequantize_strided_and_odd():
    for k in (1, 7, 33, 100, 1000):
        q, s = m4.coded(9, k, seed=k)
        wide_q = torch.zeros((9, q.shape[1] + 5), dtype=torch.uint8).cuda()
        wide_s = torch.zeros((9, s.shape[1] + 3), dtype=torch.uint8).cuda()
        wide_q[:, 3:3 + q.shape[1]], wide_s[:, 1:1 + s.shape[1]] = q.cuda(), s.cuda()
        out = torch.full((9, k + 9), 7.0, device="cuda")
        y = out[:, 2:2 + k]
        assert qmm.mx4_dequantize(wide_q[:, 3:3 + q.shape[1]], wide_s[:, 1:1 + s.shape[1]], k, out=y) is y
        assert torch.equal(y.cpu().double(), m4.values_ref(q, s, k))
        assert (out[:, :2] == 7).all() and (out[:, 2 + k:] == 7).all()


# ------------------------------------------------------------------ the packed layout
@pytest.mark.parametrize("e,n,k", [(1, 1, 1), (1, 16, 128), (3, 17, 96), (2, 40, 513), (1, 33, 2048), (2, 5, 700)])
def test_pack_by_the_header(e, n, k):
    """Every byte where the header says."""
    q, s = m4.coded(e * n, k, seed=n + k, lo=0, hi=255)
    B = m4.blocks(k)
    W = qmm.mx4_pack(q.view(e, n, -1).cuda(), s.view(e, n, -1).cuda())
    strips, C = -(-n // 16), -(-k // 512)
    W = W.cpu().view(e, strips, C, 4352)
    codes = torch.zeros((e, strips, 16, C, 4, 4, 16), dtype=torch.uint8)  # column, chunk, block / 4, block % 4, byte
    scales = torch.full((e, strips, 16, C, 4, 4), 127, dtype=torch.uint8)
    for i in range(e):
        for j in range(n):
            codes[i, j // 16, j % 16].view(16 * C, 16)[:B] = q[i * n + j].view(B, 16)
            scales[i, j // 16, j % 16].view(16 * C)[:B] = s[i * n + j]
    assert torch.equal(W[..., :4096].reshape(e, strips, C, 4, 4, 16, 16), codes.permute(0, 1, 3, 5, 4, 2, 6))
    assert torch.equal(W[..., 4096:].reshape(e, strips, C, 4, 16, 4), scales.permute(0, 1, 3, 4, 2, 5))
    two = qmm.mx4_pack(q[:n].cuda(), s[:n].cuda())
    assert torch.equal(two.cpu(), W[0].flatten())


def test_pack_takes_any_alignment():
    q, s = m4.coded(20, 200, seed=1)
    wq, ws = torch.zeros((20, q.shape[1] + 7), dtype=torch.uint8).cuda(), torch.zeros((20, 12), dtype=torch.uint8).cuda()
    wq[:, 3:3 + q.shape[1]], ws[:, 1:8] = q.cuda(), s.cuda()
    assert torch.equal(qmm.mx4_pack(wq[:, 3:3 + q.shape[1]], ws[:, 1:8]), qmm.mx4_pack(q.cuda(), s.cuda()))


# ------------------------------------------------------------------ product
SIZES = [(1, 1, 1), (1, 17, 33), (1, 300, 1024), (2, 64, 4096), (3, 64, 64), (4, 1000, 2050), (5, 100, 257),
         (8, 96, 528), (15, 48, 3000), (16, 130, 1000), (17, 33, 128), (33, 515, 260), (64, 256, 512),
         (65, 129, 300), (100, 1024, 96), (200, 70, 96), (257, 260, 784), (300, 520, 1040), (513, 700, 2064),
         (2100, 2100, 300), (2300, 1900, 145), (4090, 1030, 1024), (2950, 2900, 145), (1500, 2900, 200),
         (4, 48, 16384), (1, 40, 65536), (2, 20, 40000), (16, 36, 16400), (40, 36, 20000), (16, 4100, 512),
         # blocks of 64 rows: 2 and 4 strips a workgroup; tiles of 128 and 256 that are not whole
         (70, 4000, 300), (257, 1400, 784), (600, 1200, 260), (16000, 20, 96), (900, 1200, 270), (1111, 1000, 1040),
         (1300, 2000, 96), (3500, 3600, 150), (3330, 4000, 600)]


def weights(n, k, seed):
    q, s = m4.weight(n, k, seed)
    return qmm.mx4_pack(q.cuda(), s.cuda()), m4.values_ref(q, s)


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("kind,out", [("codes", "fp32"), ("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32")])
def test_gemm(m, n, k, kind, out):
    W, wv = weights(n, k, n + 7)
    if kind == "codes":
        q, s = m4.coded(m, k, m + k, 120, 130)
        y = qmm.mx4_gemm(q.cuda(), W, n, sx=m4.padded(s), out_dtype=TYPES[out])
    else:
        x = m4.tokens(m, k, m + n + k, TYPES[kind])
        q, s = m4.quantize_ref(x)
        y = qmm.mx4_gemm(x.cuda(), W, n, out_dtype=TYPES[out])
    assert y.dtype == TYPES[out]
    xv = m4.values_ref(q, s)
    m4.assert_close(y, xv @ wv.t(), m4.gemm_bound(xv, wv, TYPES[out]), f"gemm {m} {n} {k}")


# rows (few, up to 64, blocks of 64, tiles of 128 and of 256) and columns
SHAPES = [(1, 50), (3, 50), (16, 50), (50, 50), (130, 50), (300, 50), (1000, 1100), (3500, 3500)]


@pytest.mark.parametrize("m,n", SHAPES)
@pytest.mark.parametrize("k", [128, 160, 512, 900, 2048])
def test_whole_sums_are_exact(m, n, k):
    """Scales of 1: every sum is a whole multiple of a quarter below 2^24 quarters; each block in its place
    (the codes of a block depend on it)."""
    g = torch.Generator().manual_seed(m + k)
    B = m4.blocks(k)
    c = torch.randint(0, 16, (m, 32 * B), generator=g, dtype=torch.uint8)
    d = torch.randint(0, 16, (n, 32 * B), generator=g, dtype=torch.uint8)
    one = lambda r: torch.full((r, B), 127, dtype=torch.uint8)  # noqa: E731
    W = qmm.mx4_pack(m4.pack(d).cuda(), one(n).cuda())
    y = qmm.mx4_gemm(m4.pack(c).cuda(), W, n, sx=m4.padded(one(m))).cpu().double()
    assert torch.equal(y, m4.VALUES[c.long()] @ m4.VALUES[d.long()].t())


@pytest.mark.parametrize("m,n", [(1, 37), (7, 37), (40, 37), (150, 37), (1000, 1100), (3500, 3500)])
def test_one_block_at_a_time(m, n):
    """One block of x and one of W are not zero, each with a scale of its own: the product of the pair, exactly,
    wherever they meet, for every place of a row."""
    k = 1184
    B = m4.blocks(k)
    for b in range(B) if m < 1000 else (0, 7, 15, 16, 30, 36):
        c = torch.zeros((m, 32 * B), dtype=torch.uint8)
        d = torch.zeros((n, 32 * B), dtype=torch.uint8)
        g = torch.Generator().manual_seed(b)
        c[:, 32 * b:32 * b + 32] = torch.randint(0, 16, (m, 32), generator=g, dtype=torch.uint8)
        d[:, 32 * b:32 * b + 32] = torch.randint(0, 16, (n, 32), generator=g, dtype=torch.uint8)
        sc = torch.randint(0, 200, (m, B), generator=g, dtype=torch.uint8)
        sd = torch.randint(0, 200, (n, B), generator=g, dtype=torch.uint8)
        sc[:, b], sd[:, b] = 100 + torch.arange(m) % 20, 120 + torch.arange(n) % 17
        y = qmm.mx4_gemm(m4.pack(c).cuda(), qmm.mx4_pack(m4.pack(d).cuda(), sd.cuda()), n, sx=m4.padded(sc)).cpu().double()
        want = (m4.VALUES[c.long()] @ m4.VALUES[d.long()].t()) * m4.scale_ref(sc)[:, b:b + 1] * m4.scale_ref(sd)[:, b]
        assert torch.equal(y, want), b


@pytest.mark.parametrize("m,n", [(1, 70), (6, 70), (40, 70), (90, 70), (300, 70), (1000, 1100), (3500, 3500)])
def test_gemm_strided(m, n):
    k = 200
    W, wv = weights(n, k, 3)
    q, s = m4.coded(2 * m, k, 5, 120, 130)
    big = torch.full((2 * m, q.shape[1] + 48), 255, dtype=torch.uint8).cuda()
    big[:, 16:16 + q.shape[1]] = q.cuda()
    sb = torch.full((2 * m, 24), 255, dtype=torch.uint8).cuda()
    sb[:, 8:8 + s.shape[1]] = s.cuda()
    xv = m4.values_ref(q, s)[::2]
    ref = xv @ wv.t()
    for t, at in ((torch.float32, 0), (torch.float32, 1), (torch.bfloat16, 8), (torch.float16, 3)):
        out = torch.full((m, n + 33), 7.0, dtype=t, device="cuda")
        y = out[:, at:at + n]
        assert qmm.mx4_gemm(big[::2, 16:16 + q.shape[1]], W, n, sx=sb[::2, 8:8 + s.shape[1]], out=y) is y
        m4.assert_close(y, ref, m4.gemm_bound(xv, wv, t), f"strided {t} {at}")
        keep = torch.ones(n + 33, dtype=torch.bool)
        keep[at:at + n] = False
        assert (out.cpu()[:, keep] == 7.0).all()
    x = m4.tokens(m, 400, 9, torch.bfloat16).cuda()
    for v in (x[:, 3:203], x[:, 8:208], x[:, 200:]):
        xq = m4.values_ref(*m4.quantize_ref(v.cpu()))
        m4.assert_close(qmm.mx4_gemm(v, W, n), xq @ wv.t(), m4.gemm_bound(xq, wv, torch.float32), "strided x")


@pytest.mark.parametrize("m,n", [(1, 50), (5, 50), (20, 50), (100, 50), (300, 50), (1000, 1100), (3500, 3500)])
def test_rows_that_are_not_finite_touch_no_other(m, n):
    k = 300
    W, _ = weights(n, k, 2)
    x = m4.tokens(m, k, seed=1, dtype=torch.bfloat16)
    clean = qmm.mx4_gemm(x.cuda(), W, n).cpu()
    x[m // 2, 299] = math.inf
    y = qmm.mx4_gemm(x.cuda(), W, n).cpu()
    assert torch.isnan(y[m // 2]).all()
    y[m // 2] = clean[m // 2]
    assert torch.equal(y, clean)
    # a weight's row
    q, s = m4.weight(n, k, 2)
    s[3, 4] = 255
    y = qmm.mx4_gemm(m4.tokens(m, k, seed=1, dtype=torch.bfloat16).cuda(), qmm.mx4_pack(q.cuda(), s.cuda()), n).cpu()
    assert torch.isnan(y[:, 3]).all()
    y[:, 3] = clean[:, 3]
    assert torch.equal(y, clean)


def test_empty():
    W, _ = weights(16, 64, 1)
    assert qmm.mx4_gemm(torch.zeros((0, 64), device="cuda"), W, 16).shape == (0, 16)
    none = torch.zeros(0, dtype=torch.uint8, device="cuda")
    y = qmm.mx4_gemm(torch.zeros((3, 0), device="cuda"), none, 16, out=torch.full((3, 16), 7.0, device="cuda"))
    assert (y == 0).all()
    assert qmm.mx4_gemm(torch.zeros((3, 64), device="cuda"), none, 0).shape == (3, 0)
    q, s = qmm.mx4_quantize(torch.zeros((3, 0), device="cuda"))
    assert q.shape == (3, 0) and s.shape == (3, 0) and qmm.mx4_dequantize(q, s).shape == (3, 0)


# ------------------------------------------------------------------ mixture of experts
def experts(e, d, i, seed):
    """Packed weights and values of e experts' three weights."""
    packed, values = [], []
    for j, (n, k) in enumerate(((i, d), (i, d), (d, i))):
        qs = [m4.weight(n, k, seed + 100 * x + j) for x in range(e)]
        packed.append(qmm.mx4_pack(torch.stack([q for q, _ in qs]).cuda(), torch.stack([s for _, s in qs]).cuda()))
        values.append(torch.stack([m4.values_ref(q, s, k) for q, s in qs]))
    return packed, values


# (T, D, I, E, top_k): single elements; below, at and across strips of 16, steps of 128 and chunks of 512;
# tokens in 1 to 4 row tiles; all experts for all; more places than experts and fewer
MOE = [(1, 1, 1, 1, 1), (1, 64, 64, 4, 2), (1, 512, 300, 40, 8), (2, 33, 17, 3, 3), (5, 100, 77, 6, 3),
       (8, 700, 515, 5, 1), (16, 256, 128, 8, 2), (17, 130, 200, 8, 2), (33, 96, 1040, 4, 4), (64, 256, 128, 16, 6),
       (3, 2056, 48, 130, 8), (64, 40, 40, 2, 1), (7, 128, 2050, 70, 5)]


@pytest.mark.parametrize("T,D,I,E,k", MOE)
@pytest.mark.parametrize("x,out,act,norm", [("bf16", "bf16", "silu", True), ("fp16", "fp32", "gelu", False),
                                            ("fp32", "fp16", "gelu_tanh", True), ("fp32", "fp32", "silu", False)])
def test_moe(T, D, I, E, k, x, out, act, norm):
    packed, values = experts(E, D, I, T + D)
    v = m4.tokens(T, D, seed=I, dtype=TYPES[x])
    lg = torch.randn((T, E), generator=torch.Generator().manual_seed(k)) * 2
    y = qmm.mx4_moe(v.cuda(), *packed, I, logits=lg.cuda(), top_k=k, renormalize=norm, act=act, out_dtype=TYPES[out])
    assert y.dtype == TYPES[out]
    ref, bound = m4.moe_ref(act, v, *values, *m4.route_ref(lg, k, norm), TYPES[out])
    m4.assert_close(y, ref, bound, f"moe {T} {D} {I} {E} {k}")


# (T, D, I, E, top_k, n): tiles enough, of E experts' weights, for workgroups that hold an expert's rows: in the first half,
# the second, both, the second in ranges; n experts alone are chosen, so that more of one's tokens come than are held at once
MANY = [(64, 130, 330, 300, 8, 60), (64, 460, 40, 300, 8, 60), (64, 460, 330, 260, 8, 9), (16, 460, 330, 256, 32, 33),
        (8, 460, 330, 256, 32, 40), (4, 897, 650, 128, 32, 34), (64, 2100, 330, 260, 8, 16), (64, 460, 2100, 260, 8, 16),
        (20, 4000, 330, 300, 32, 40), (16, 900, 9000, 40, 8, 4)]


@pytest.mark.parametrize("T,D,I,E,k,n", MANY)
@pytest.mark.parametrize("x,out", [("bf16", "fp16"), ("fp16", "fp32"), ("fp32", "bf16"), ("fp32", "fp32")])
def test_moe_of_many_tiles(T, D, I, E, k, n, x, out):
    some, values = experts(n, D, I, T + D)
    g = torch.Generator().manual_seed(k)
    of = torch.sort(torch.randperm(E, generator=g)[:n]).values
    packed = []
    for w in some:
        packed.append(torch.zeros((E,) + tuple(w.shape[1:]), dtype=torch.uint8, device="cuda"))
        packed[-1][of.cuda()] = w
    v = m4.tokens(T, D, seed=I, dtype=TYPES[x])
    lg = torch.randn((T, n), generator=g) * 2
    full = torch.full((T, E), -math.inf)
    full[:, of] = lg
    y = qmm.mx4_moe(v.cuda(), *packed, I, logits=full.cuda(), top_k=k, out_dtype=TYPES[out])
    ref, bound = m4.moe_ref("silu", v, *values, *m4.route_ref(lg, k, True), TYPES[out])
    m4.assert_close(y, ref, bound, f"moe {T} {D} {I} {E} {k} {n}")


# few tokens: rows of whole 16 bytes and others, h that fits a workgroup's LDS and one that does not, more than 64 places
FEW = [(1, 8, 40, 4, 4), (2, 520, 520, 9, 3), (3, 1032, 77, 128, 8), (4, 2064, 300, 16, 16), (4, 72, 96, 40, 17), (4, 40, 2600, 20, 5),
       (4, 64, 96, 300, 32), (1, 512, 8200, 2, 2), (2, 4104, 64, 3, 1), (8, 72, 96, 300, 32), (5, 1001, 77, 16, 4), (7, 33, 50, 40, 17),
       (8, 2600, 40, 100, 9)]


@pytest.mark.parametrize("T,D,I,E,k", FEW)
@pytest.mark.parametrize("x,out,norm", [("bf16", "bf16", True), ("fp16", "fp32", True), ("fp32", "fp16", False), ("fp32", "fp32", True)])
def test_moe_few_tokens(T, D, I, E, k, x, out, norm):
    packed, values = experts(E, D, I, T + D)
    v = m4.tokens(T, D, seed=I, dtype=TYPES[x])
    lg = torch.randn((T, E), generator=torch.Generator().manual_seed(k)) * 2
    y = qmm.mx4_moe(v.cuda(), *packed, I, logits=lg.cuda(), top_k=k, renormalize=norm, out_dtype=TYPES[out])
    ref, bound = m4.moe_ref("silu", v, *values, *m4.route_ref(lg, k, norm), TYPES[out])
    m4.assert_close(y, ref, bound, f"moe {T} {D} {I} {E} {k}")
    # experts given, the first of them twice
    ids = torch.randint(0, E, (T, k), generator=torch.Generator().manual_seed(D), dtype=torch.int32)
    ids[:, -1] = ids[:, 0]
    w = torch.randn((T, k), generator=torch.Generator().manual_seed(I))
    y = qmm.mx4_moe(v.cuda(), *packed, I, ids=ids.cuda(), weights=w.cuda(), out_dtype=TYPES[out])
    ref, bound = m4.moe_ref("silu", v, *values, ids, w, TYPES[out])
    m4.assert_close(y, ref, bound, f"given {T} {D} {I} {E} {k}")


@pytest.mark.parametrize("T", [1, 4, 20, 64])
@pytest.mark.parametrize("itype", [torch.int32, torch.int64])
def test_moe_given_experts(T, itype):
    """Ids outside the range, the same expert twice, rows without any; weights of every type, zero and negative."""
    D, I, E, k = 160, 100, 7, 4
    packed, values = experts(E, D, I, 5)
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(-2, E + 2, (T, k), generator=g).to(itype)
    ids[0] = torch.tensor([3, -1, 3, E])
    if T > 2:
        ids[1], ids[2] = -1, torch.iinfo(itype).max
        ids[3] = 2
    if itype == torch.int64:
        ids[0, 1] = (1 << 32) + 1  # an expert in its low bits alone
    for wt in TYPES.values():
        w = torch.randn((T, k), generator=g).to(wt)
        w[-1, -1] = 0.0
        v = m4.tokens(T, D, seed=1, dtype=torch.bfloat16)
        y = qmm.mx4_moe(v.cuda(), *packed, I, ids=ids.cuda(), weights=w.cuda())
        ref, bound = m4.moe_ref("silu", v, *values, ids, w, torch.float32)
        m4.assert_close(y, ref, bound, f"given {T} {wt}")
        if T > 2:
            assert (y[1:3] == 0).all()


@pytest.mark.parametrize("T,E,k", [(64, 1, 32), (3, 1, 5), (64, 2, 17), (4, 2, 16)])
def test_moe_more_places_than_experts(T, E, k):
    D, I = 72, 40
    packed, values = experts(E, D, I, 4)
    g = torch.Generator().manual_seed(T)
    ids, w = torch.randint(-1, E + 1, (T, k), generator=g), torch.randn((T, k), generator=g)
    v = m4.tokens(T, D, seed=1, dtype=torch.bfloat16)
    y = qmm.mx4_moe(v.cuda(), *packed, I, ids=ids.cuda(), weights=w.cuda())
    ref, bound = m4.moe_ref("silu", v, *values, ids, w, torch.float32)
    m4.assert_close(y, ref, bound, f"places {T} {E} {k}")


@pytest.mark.parametrize("lt", TYPES)
def test_moe_equal_logits_take_the_lowest(lt):
    T, D, I, E, k = 20, 64, 48, 150, 5
    packed, values = experts(E, D, I, 9)
    lg = torch.randint(-2, 3, (T, E), generator=torch.Generator().manual_seed(0)).to(TYPES[lt])
    lg[0] = 0.0
    lg[1, ::2] = -0.0
    lg[1, 1::2] = 0.0
    v = m4.tokens(T, D, seed=1)
    y = qmm.mx4_moe(v.cuda(), *packed, I, logits=lg.cuda(), top_k=k)
    ref, bound = m4.moe_ref("silu", v, *values, *m4.route_ref(lg, k, True), torch.float32)
    m4.assert_close(y, ref, bound, "ties")


@pytest.mark.parametrize("norm", [True, False])
def test_moe_logits_at_their_ends(norm):
    """Minus infinities (fewer than k left, none left), far apart, the lowest value, NaN and infinity."""
    T, D, I, E, k = 9, 64, 48, 10, 4
    packed, values = experts(E, D, I, 2)
    lg = torch.randn((T, E), generator=torch.Generator().manual_seed(0))
    lg[0] = -math.inf
    lg[1, 2:] = -math.inf
    lg[2] = torch.linspace(-300, 300, E)
    lg[3] = torch.finfo(torch.float32).min
    lg[4, 3:] = torch.finfo(torch.float32).min
    lg[5, 5] = 3e38
    lg[6, 1] = math.nan
    lg[7, 4] = math.inf
    v = m4.tokens(T, D, seed=1)
    y = qmm.mx4_moe(v.cuda(), *packed, I, logits=lg.cuda(), top_k=k, renormalize=norm).cpu()
    assert (y[0] == 0).all() and torch.isnan(y[6]).all() and torch.isnan(y[7]).all()
    ok = [1, 2, 3, 4, 5, 8]
    ref, bound = m4.moe_ref("silu", v[ok], *values, *m4.route_ref(lg[ok], k, norm), torch.float32)
    m4.assert_close(y[ok], ref, bound, "ends")


@pytest.mark.parametrize("T", [3, 40])
def test_moe_strided(T):
    D, I, E, k = 90, 70, 6, 2
    packed, values = experts(E, D, I, 2)
    base, lb = m4.tokens(2 * T, 200, 1, torch.float16).cuda(), torch.randn((T, 30), generator=torch.Generator().manual_seed(3)).cuda()
    for at, t in ((0, torch.float32), (1, torch.float16), (8, torch.bfloat16)):
        out = torch.full((T, D + 40), 7.0, dtype=t, device="cuda")
        v, lg, y = base[::2, at:at + D], lb[:, at:at + E], out[:, at:at + D]
        assert qmm.mx4_moe(v, *packed, I, logits=lg, top_k=k, out=y) is y
        ref, bound = m4.moe_ref("silu", v.cpu(), *values, *m4.route_ref(lg.cpu(), k, True), t)
        m4.assert_close(y, ref, bound, "strided")
        assert (out[:, :at] == 7).all() and (out[:, at + D:] == 7).all()


@pytest.mark.parametrize("T", [2, 30])
def test_moe_not_finite_stays_in_its_row(T):
    D, I, E, k = 96, 70, 4, 2
    packed, values = experts(E, D, I, 2)
    lg = torch.randn((T, E), generator=torch.Generator().manual_seed(3)).cuda()
    for t in TYPES.values():
        v = m4.tokens(T, D, seed=1, dtype=t)
        clean = qmm.mx4_moe(v.cuda(), *packed, I, logits=lg, top_k=k).cpu()
        for bad in (math.nan, math.inf, -math.inf):
            b = v.clone()
            b[T - 1, D - 1] = bad
            y = qmm.mx4_moe(b.cuda(), *packed, I, logits=lg, top_k=k).cpu()
            assert torch.isnan(y[T - 1]).all() and torch.equal(y[:T - 1], clean[:T - 1])


def test_moe_empty():
    packed, _ = experts(2, 64, 32, 1)
    z = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    assert qmm.mx4_moe(z(0, 64), *packed, 32, logits=z(0, 2), top_k=1).shape == (0, 64)
    none = torch.zeros((3, 0), dtype=torch.int32, device="cuda")
    y = qmm.mx4_moe(z(3, 64), *packed, 32, ids=none, weights=z(3, 0), out=torch.full((3, 64), 7.0, device="cuda"))
    assert (y == 0).all()
    zero = torch.zeros((0, 0), dtype=torch.uint8, device="cuda")
    y = qmm.mx4_moe(z(3, 64), zero, zero, zero, 32, logits=z(3, 0), top_k=0, out=torch.full((3, 64), 7.0, device="cuda"))
    assert (y == 0).all()


# ------------------------------------------------------------------ together, graphs, streams
def layer(x, packed, I, W, n, lg, k):
    """A mixture, then a product on the same format."""
    h = qmm.mx4_moe(x, *packed, I, logits=lg, top_k=k, out_dtype=x.dtype)
    return qmm.mx4_gemm(h, W, n, out_dtype=x.dtype)


def test_run_together_from_quantizer_to_product():
    T, D, I, E, k, n = 12, 256, 200, 6, 2, 90
    g = torch.Generator().manual_seed(1)
    w = [[torch.randn(s, generator=g) / math.sqrt(s[1]) for _ in range(E)] for s in ((I, D), (I, D), (D, I))]
    wn = torch.randn((n, D), generator=g) / 16
    coded = [[qmm.mx4_quantize(v.cuda()) for v in part] for part in w]
    packed = [qmm.mx4_pack(torch.stack([q for q, _ in part]), torch.stack([s for _, s in part])) for part in coded]
    values = [torch.stack([qmm.mx4_dequantize(q, s, v.shape[1]).cpu().double() for (q, s), v in zip(c, part)])
              for c, part in zip(coded, w)]
    W = qmm.mx4_pack(*qmm.mx4_quantize(wn.cuda()))
    x, lg = m4.tokens(T, D, 2, torch.bfloat16), torch.randn((T, E), generator=g)
    y = layer(x.cuda(), packed, I, W, n, lg.cuda(), k)
    h = qmm.mx4_moe(x.cuda(), *packed, I, logits=lg.cuda(), top_k=k, out_dtype=torch.bfloat16)
    ref, bound = m4.moe_ref("silu", x, *values, *m4.route_ref(lg, k, True), torch.bfloat16)
    m4.assert_close(h, ref, bound, "mixture")
    hv = m4.values_ref(*m4.quantize_ref(h.cpu()))
    wv = m4.values_ref(*m4.quantize_ref(wn))
    m4.assert_close(y, hv @ wv.t(), m4.gemm_bound(hv, wv, torch.bfloat16), "product")


@pytest.mark.parametrize("T", [1, 20, 64])
def test_graph_replays_between_eager_calls(T):
    D, I, E, k, n = 256, 200, 6, 2, 90
    packed, _ = experts(E, D, I, 2)
    W, _ = weights(n, D, 3)
    x, lg = torch.zeros((T, D), device="cuda", dtype=torch.bfloat16), torch.zeros((T, E), device="cuda")
    layer(x, packed, I, W, n, lg, k)
    torch.cuda.synchronize()
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer(x, packed, I, W, n, lg, k)
    with torch.cuda.graph(other):
        y2 = layer(x, packed, I, W, n, lg, k)
    for i in range(5):
        g = torch.Generator().manual_seed(i)
        x.copy_(m4.tokens(T, D, i, torch.bfloat16))
        lg.copy_(torch.randn((T, E), generator=g))
        want = layer(x, packed, I, W, n, lg, k)
        graph.replay()
        other.replay()
        layer(x[:1], packed, I, W, n, lg[:1], k)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(y2, want)


@pytest.mark.parametrize("T,D,I,E,k,n", [(64, 460, 330, 260, 8, 13), (16, 900, 9000, 40, 8, 4), (5, 72, 96, 300, 32, 3),
                                         (3, 77, 2600, 40, 20, 4)])
def test_forms_replayed_and_on_two_streams_at_once(T, D, I, E, k, n):
    """Held rows, ranges of them, rows through LDS, few tokens: n experts' weights, E / n times."""
    packed = [w.repeat(E // n, 1) for w in experts(n, D, I, 5)[0]]
    x, lg = torch.zeros((T, D), device="cuda", dtype=torch.float16), torch.zeros((T, E), device="cuda")
    call = lambda: qmm.mx4_moe(x, *packed, I, logits=lg, top_k=k, renormalize=False, act="gelu")  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = call()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(4):
        g = torch.Generator().manual_seed(i)
        x.copy_(m4.tokens(T, D, i, torch.float16))
        lg.copy_(torch.randn((T, E), generator=g))
        want = call()
        graph.replay()
        call()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        got = []
        for _ in range(3):
            for s in streams:
                with torch.cuda.stream(s):
                    got.append(call())
        torch.cuda.synchronize()
        assert all(torch.equal(v, want) for v in got)


def test_other_stream_and_run_to_run():
    T, D, I, E, k, n = 33, 700, 300, 8, 3, 500
    packed, _ = experts(E, D, I, 2)
    W, _ = weights(n, D, 3)
    x, lg = m4.tokens(T, D, 1, torch.bfloat16).cuda(), torch.randn((T, E), generator=torch.Generator().manual_seed(1)).cuda()
    want = layer(x, packed, I, W, n, lg, k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [layer(x, packed, I, W, n, lg, k) for _ in range(4)]
    s.synchronize()
    for g in got:
        assert torch.equal(g, want)


@pytest.mark.parametrize("m", [3, 20, 70, 300, 6000])
def test_a_row_does_not_depend_on_its_neighbours(m):
    n, k = 200, 1000
    W, _ = weights(n, k, 1)
    x = m4.tokens(m, k, 2, torch.bfloat16).cuda()
    whole = qmm.mx4_gemm(x, W, n)
    xv = m4.values_ref(*m4.quantize_ref(x.cpu()))
    q, s = m4.weight(n, k, 1)
    bound = m4.gemm_bound(xv, m4.values_ref(q, s), torch.float32)
    for i in (0, m // 2, m - 1):
        alone = qmm.mx4_gemm(x[i:i + 1], W, n)
        assert ((alone - whole[i:i + 1]).abs().cpu().double() <= 2 * bound[i:i + 1]).all()


def test_warns_where_gradients_end():
    x = torch.zeros((2, 64), device="cuda", requires_grad=True)
    with pytest.warns(UserWarning, match="passes none on"):
        qmm.mx4_quantize(x)
    with torch.no_grad():
        qmm.mx4_quantize(x)


def test_example_runs():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mx4_experts.py")
    spec = importlib.util.spec_from_file_location("mx4_experts", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    for tokens in ("1", "6", "40"):
        assert all(mod.main(["--width", "512", "--hidden", "160", "--experts", "12", "--top-k", "3", "--vocab", "1000",
                             "--tokens", tokens], log=lambda *_: None))
