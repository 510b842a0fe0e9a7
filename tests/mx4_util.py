"""Inputs, 64-bit references and error bounds for the microscaled 4-bit operators."""
import math

import torch

from int8_util import TYPES, U, act_ref, assert_close, half, round_bound, tiny  # noqa: F401

VALUES = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def blocks(k):
    return -(-k // 32)


def unpack(codes):
    """One code per element of bytes that hold two."""
    return torch.stack([codes & 15, codes >> 4], -1).flatten(-2)


def pack(c):
    return c[..., 0::2] | (c[..., 1::2] << 4)


def quantize_ref(x):
    """(codes, scales) by the definition, from exponents and borders in 64 bits."""
    m, k = x.shape
    v = torch.zeros((m, blocks(k) * 32), dtype=torch.float64)
    v[:, :k] = x.double()
    v = v.reshape(m, blocks(k), 32)
    bad = ~torch.isfinite(v).all(2)
    v = torch.where(bad[:, :, None], torch.zeros_like(v), v)
    top = v.abs().amax(2)
    e = torch.where(top > 0, torch.frexp(top)[1] - 3, torch.full(top.shape, -127)).clamp(min=-127)
    a = v.abs() * torch.ldexp(torch.ones_like(top), -e)[:, :, None]
    # the code's neighbours by value: nearest, ties to the even code
    grid = VALUES[:8]
    d = (a[..., None] - grid).abs()
    near = d.min(-1).values
    even = torch.tensor([0, 2, 4, 6])
    is_even = (d[..., even] == near[..., None])
    c = torch.where(is_even.any(-1), even[is_even.int().argmax(-1)], d.argmin(-1))
    c = c + 8 * torch.signbit(v).long()
    c = torch.where(bad[:, :, None], torch.zeros_like(c), c)
    e = torch.where(bad, torch.full_like(e, 128), e)
    return pack(c.reshape(m, 32 * blocks(k)).to(torch.uint8)), (e + 127).to(torch.uint8)


def scale_ref(s):
    v = torch.ldexp(torch.ones(s.shape, dtype=torch.float64), s.int() - 127)
    return torch.where(s == 255, torch.full_like(v, math.nan), v)


def values_ref(codes, scales, k=None):
    v = VALUES[unpack(codes).long()]
    v = (v.unflatten(-1, (-1, 32)) * scale_ref(scales)[..., None]).flatten(-2)
    return v if k is None else v[..., :k]


def coded(n, k, seed, lo=110, hi=125):
    """Random codes and scales; codes past k are zeros, as the quantizer leaves them."""
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(0, 16, (n, blocks(k) * 32), generator=g, dtype=torch.uint8)
    c[:, k:] = 0
    return pack(c), torch.randint(lo, hi + 1, (n, blocks(k)), generator=g, dtype=torch.uint8)


def tokens(m, k, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((m, k), generator=g)
    if k > 3:
        x[:, k // 3] *= 16.0
    return x.to(dtype)


def weight(n, k, seed):
    """Codes and scales of a normal weight with rows of about unit length."""
    g = torch.Generator().manual_seed(seed)
    return quantize_ref(torch.randn((n, k), generator=g) / math.sqrt(max(k, 1)))


def padded(s):
    """Scales as a view of rows of whole 4 bytes, the padding NaN's byte (it may not count)."""
    whole = torch.full((s.shape[0], max(4, -(-s.shape[1] // 4) * 4)), 255, dtype=torch.uint8)
    whole[:, :s.shape[1]] = s
    return whole.cuda()[:, :s.shape[1]]


def gemm_bound(x, w, t):
    """Of sums of |x w| = a.  A block's products (32, multiples of a quarter below 2^11) are summed
    exactly; each step adds 4 blocks to the accumulator, aligned to the largest of the 5 and cut off below
    its last bits: 5 U each of at most a, twice that for a cut instead of a rounding; waves or splits
    (at most 16) add 16 more roundings.  Then y's rounding."""
    ref = x @ w.t()
    steps = -(-x.shape[1] // 128)
    return (x.abs() @ w.abs().t()) * (10 * steps + 16) * U + round_bound(ref, t) + 2.0 ** -126


# ------------------------------------------------------------------ mixture of experts
def route_ref(logits, k, renormalize):
    """ids and weights in 64 bits: the k largest, the lower index of equal ones, no -inf."""
    lg = logits.double()
    top, ids = torch.sort(lg, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    ex = torch.exp(top - top[:, :1])
    of = ex.sum(1, keepdim=True) if renormalize else torch.exp(lg - top[:, :1]).sum(1, keepdim=True)
    gone = torch.isneginf(top)
    return torch.where(gone, torch.full_like(ids, -1), ids), torch.where(gone, torch.zeros_like(ex), ex / of)


def moe_ref(act, x, wg, wu, wd, ids, w, t):
    """y in 64 bits and a bound of what 32 bits make of it.  wg, wu, wd: values (E, ., .)."""
    T, D = x.shape
    E, I = wg.shape[0], wg.shape[1]
    x = x.double()
    y, b = torch.zeros((T, D), dtype=torch.float64), torch.zeros((T, D), dtype=torch.float64)
    # a sum of K products of exact bf16 values in fp32: K roundings (cut off: 2) at most, and 16 of waves
    sum_u, sum_d = (2 * D + 16) * U, (2 * I * ids.shape[1] + 16) * U
    # h keeps 24 bits (3 parts) for fp32 y, else 16 (2 parts: 8 cut off and 8 rounded)
    part = 2 * U if t == torch.float32 else 2.0 ** -16
    for i in range(T):
        for j in range(ids.shape[1]):
            e = int(ids[i, j])
            if e < 0 or e >= E:
                continue
            g, u = wg[e] @ x[i], wu[e] @ x[i]
            eg, eu = (wg[e].abs() @ x[i].abs()) * sum_u, (wu[e].abs() @ x[i].abs()) * sum_u
            a, da, amp = act_ref(act, g)
            # |act'| is at most 1.13; the evaluation's own part as in int8_util.gated_bound
            ea = 1.2 * eg + a.abs() * (40 + 16 * amp) * U + 2.0 ** -120
            h = a * u
            eh = ea * u.abs() + (a.abs() + ea) * eu
            wt = float(w[i, j])
            y[i] += wt * (wd[e] @ h)
            # the weight itself: exponentials and a quotient, 40 U with exponents to 16
            b[i] += abs(wt) * (wd[e].abs() @ (eh + h.abs() * (part + sum_d + 64 * U)))
    return y, b + round_bound(y, t) + 2.0 ** -120
