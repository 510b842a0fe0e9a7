"""Inputs, 64-bit references and error bounds for the int8 x int8 operators.

The bounds count roundings.  `half(t)` is the relative error of one rounding
to type t (half a step, eps / 2); `tiny(t)` the absolute one among subnormals.
fp32 steps are counted in units of U = 2^-24.
"""
import math

import torch

U = 2.0 ** -24
TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def half(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    return {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -149}[t]


def pad16(k):
    return -(-k // 16) * 16


def codes(rows, k, g, lo=-127, hi=127):
    """int8 codes (rows, k) as a view of rows padded to 16 bytes; the padding
    holds codes too, which may not count."""
    return torch.randint(lo, hi + 1, (rows, max(16, pad16(k))), generator=g, dtype=torch.int8)[:, :k]


def weight(n, k, seed, lo=-128, hi=127):
    g = torch.Generator().manual_seed(seed)
    return codes(n, k, g, lo, hi), (0.5 + torch.rand(n, generator=g)) / (60.0 * math.sqrt(max(k, 1)))


def tokens(m, k, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((m, k), generator=g)
    if k > 3:
        x[:, k // 3] *= 16.0
    return x.to(dtype)


def cuda(t):
    """To the GPU with its strides and the bytes around it kept (a view of padded rows
    stays one)."""
    if t is None:
        return None
    if t.dim() == 2 and t.shape[0] > 0 and t.shape[1] != t.stride(0) and t.storage_offset() == 0:
        whole = t.as_strided((t.shape[0], t.stride(0)), (t.stride(0), 1)).cuda()
        return whole[:, :t.shape[1]]
    return t.cuda()


# ------------------------------------------------------------------ references
def quantize_ref(x):
    """(codes, scales) by the definition; the quotient in 64 bits decides every
    case that a correctly rounded 32-bit one might move to a half."""
    x = x.float()
    top = x.abs().amax(1) if x.shape[1] else torch.zeros(x.shape[0])
    s = (top.double() / 127.0).float()  # 53 bits hold enough of top / 127 to round it to 24 alike
    q = (x.double() / s.double()[:, None]).round().clamp(-127, 127)
    ok = torch.isfinite(top) & (s > 0)
    bad = ~torch.isfinite(x).all(1)
    s = torch.where(bad, torch.full_like(s, math.nan), s)
    return torch.where(ok[:, None], q, torch.zeros_like(q)).to(torch.int8), s


def act_ref(act, v):
    """act(v), act'(v), and how much a relative error of v grows in act(v)."""
    if act == "silu":
        p = torch.sigmoid(v)
        return v * p, p * (1 + v * torch.sigmoid(-v)), v.abs()
    if act == "gelu":
        p = 0.5 * torch.erfc(-v / math.sqrt(2))
        return v * p, p + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi), v * v
    c = 2 * math.sqrt(2 / math.pi)
    t = c * (v + 0.044715 * v ** 3)
    p = torch.sigmoid(t)
    return v * p, p + v * p * torch.sigmoid(-t) * c * (1 + 3 * 0.044715 * v * v), t.abs()


def product_ref(q, sx, w, sw):
    return (q.double() @ w.double().t()) * (sx.double()[:, None] * sw.double())


def round_bound(ref, t):
    return ref.abs() * (0.0 if t == torch.float32 else half(t)) + tiny(t)


def gemm_bound(ref, t):
    """The whole sum to fp32, sx sw, their product: 3 roundings; then y's."""
    return ref.abs() * 4 * U + round_bound(ref, t)


def gated_ref(act, g, u):
    a, _, amp = act_ref(act, g)
    return a * u, amp


def gated_bound(act, g, u, t):
    """g and u carry 4 U each.  act: g's error times its condition number (at most
    1 + amp, within 2), and the evaluation's own -- exponentials and quotients
    of a few U, an exponent of rounded argument again times amp: 32 + 16 amp in
    all.  u's 4 and the product's own make 8."""
    h, amp = gated_ref(act, g, u)
    # below 2^-126 the parts of the activation are subnormal or zero
    return h.abs() * (40 + 16 * amp) * U + 2.0 ** -120 * (1 + u.abs()) + round_bound(h, t)


def backward_ref(dy, q, sx, w, sw):
    d = dy.double()
    return (d * sw.double()) @ w.double(), (d * sx.double()[:, None]).t() @ q.double()


def _scale_power(s):
    m = float(s.abs().max()) if s.numel() else 0.0
    return 2.0 ** (math.frexp(m)[1]) if m > 0 else 1.0


def _product_bound(d, derr, codes_, t, power):
    """|sum d c| with d rounded to t (half a step, and tiny in units of the power of
    two taken out) on top of its own error derr, c exact: the sum in fp32 of as many
    terms, one rounding for each, and 4 for scaling."""
    n = d.shape[1]
    c = codes_.double().abs()
    return (d.abs() * (half(t) + (n + 4) * U) + derr + tiny(t) * power) @ c


def backward_bound(dy, q, sx, w, sw, t):
    d = dy.double()
    dx, dw = backward_ref(dy, q, sx, w, sw)
    zero = torch.zeros_like(d)
    bx = _product_bound(d * sw.double(), zero, w, t, _scale_power(sw))
    bw = _product_bound((d * sx.double()[:, None]).t(), zero.t(), q, t, _scale_power(sx))
    return bx + round_bound(dx, t), bw + round_bound(dw, t)


def gated_grads(act, dh, q, sx, wg, sg, wu, su):
    """dg, du in 64 bits and bounds of what fp32 makes of them."""
    g, u = product_ref(q, sx, wg, sg), product_ref(q, sx, wu, su)
    a, da, amp = act_ref(act, g)
    d = dh.double()
    # act' has no useful relative error near its zero: (64 + 32 amp) U of (1 + |g|)
    eg = (d * u).abs() * ((64 + 32 * amp) * U * (1 + g.abs()) + 8 * U * da.abs()) + 2.0 ** -120
    eu = (d * a).abs() * (48 + 16 * amp) * U + 2.0 ** -120
    return d * u * da, d * a, eg, eu


def gated_backward_ref(act, dh, q, sx, wg, sg, wu, su):
    dg, du, _, _ = gated_grads(act, dh, q, sx, wg, sg, wu, su)
    dx = (dg * sg.double()) @ wg.double() + (du * su.double()) @ wu.double()
    s = sx.double()[:, None]
    return dx, (dg * s).t() @ q.double(), (du * s).t() @ q.double()


def gated_backward_bound(act, dh, q, sx, wg, sg, wu, su, t):
    dg, du, eg, eu = gated_grads(act, dh, q, sx, wg, sg, wu, su)
    dx, dwg, dwu = gated_backward_ref(act, dh, q, sx, wg, sg, wu, su)
    pw = _scale_power(torch.cat([sg, su]))
    px = _scale_power(sx)
    s = sx.double()[:, None]
    d = torch.cat([dg * sg.double(), du * su.double()], 1)
    e = torch.cat([eg * sg.double(), eu * su.double()], 1)
    bx = _product_bound(d, e, torch.cat([wg, wu], 0), t, pw)
    bg = _product_bound((dg * s).t(), (eg * s).t(), q, t, px)
    bu = _product_bound((du * s).t(), (eu * s).t(), q, t, px)
    return bx + round_bound(dx, t), bg + round_bound(dwg, t), bu + round_bound(dwu, t)


def assert_close(got, ref, bound, what):
    """Within the bound, and finite -- but where the reference lies beyond the
    type's largest value by more than half a step, the infinity of its sign."""
    top = torch.finfo(got.dtype).max
    got = got.double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if got.numel() == 0:
        return
    over = ref.abs() - bound > top
    assert (got[over] == torch.sign(ref[over]) * math.inf).all(), f"{what}: overflow"
    got, ref, bound = got[~over], ref[~over], bound[~over]
    if got.numel() == 0:
        return
    assert torch.isfinite(got).all(), f"{what}: not finite"
    r = ((got - ref).abs() / bound.clamp(min=1e-300)).max()
    assert r <= 1.0, f"{what}: {float(r):.3g} times the bound"
