"""Mixtures whose every sum is of a term or two, so that a bound of a few roundings holds whatever D and I are: what
the kernels make of each bit of an activation shows in y.

Token t has its one value at position p[t] (two, at q too, in `pairs`); weights of the first half are any codes, a row of the
second half's has one code (two neighbours c and -c in `pairs`).
"""
import torch

import mx4_util as m4
from mx4_util import U, act_ref, round_bound


def _code(bytes_, k):
    """Codes (..., K) at positions k (last dimension indexed) of bytes (..., K / 2)."""
    b = bytes_.gather(-1, k // 2).int()
    return torch.where(k % 2 == 1, b >> 4, b & 15)


def _scale(scales, k):
    return m4.scale_ref(scales.gather(-1, k // 32).cpu())


class Terms:
    """Operands on `device` of T tokens and E experts, ids and weights (T, k) given: of each token one place counts with
    weight 1, the others with up to 1/16."""

    def __init__(self, T, D, I, E, k, dtype, pairs, seed, device):
        g = torch.Generator(device=device).manual_seed(seed)
        new = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=device)  # noqa: E731
        self.I, self.pairs = I, pairs
        byte = lambda lo, hi, *s: new(lo, hi, *s).to(torch.uint8)  # noqa: E731
        gate, up = (byte(0, 256, E, I, 16 * m4.blocks(D)) for _ in range(2))
        sg, su = (byte(121, 124, E, I, m4.blocks(D)) for _ in range(2))
        down = torch.zeros((E, D, 16 * m4.blocks(I)), dtype=torch.uint8, device=device)
        sd = byte(*((131, 139) if pairs else (118, 126)), E, D, m4.blocks(I))  # (differences are 2^-11 of terms)
        self.p = new(0, D, T)
        x = 1.0 + torch.rand((T,), generator=g, device=device, dtype=torch.float64)
        x = x * (1 - 2 * new(0, 2, T))
        v = torch.zeros((T, D), dtype=torch.float64, device=device)
        if pairs:
            # rows of two columns 2 i and 2 i + 1 of h alike but for position q, where x is 2^-11 of 8 bits
            q = D // 2
            self.q = q
            self.p = torch.where(self.p == q, (q + 1) % D, self.p)
            gate[:, 1::2], up[:, 1::2] = gate[:, 0:I - I % 2:2], up[:, 0:I - I % 2:2]
            sg[:, 1::2], su[:, 1::2] = sg[:, 0:I - I % 2:2], su[:, 0:I - I % 2:2]
            keep = 0x0F if q % 2 else 0xF0
            gate[:, :, q // 2] &= keep
            up[:, :, q // 2] &= keep
            up[:, 1::2, q // 2] |= (byte(1, 8, E, I // 2) << (4 * (q % 2)))
            x = (x * 128).round() / 128
            v[:, q] = (1.0 + new(0, 128, T).double() / 128) * 2.0 ** -11
            self.c = 2 * new(0, I // 2, E, D)
            code = byte(1, 8, E, D)
            down.scatter_(2, (self.c // 2)[:, :, None], (code | ((code + 8) << 4))[:, :, None])
        else:
            self.c = new(0, I, E, D)
            code = byte(1, 8, E, D) + 8 * byte(0, 2, E, D)
            down.scatter_(2, (self.c // 2)[:, :, None], torch.where(self.c % 2 == 1, code << 4, code)[:, :, None])
        v.scatter_(1, self.p[:, None], x[:, None])
        self.x = v.to(dtype)
        self.w = [(gate, sg), (up, su), (down, sd)]
        self.ids = torch.rand((T, E), generator=g, device=device).argsort(1)[:, :k].contiguous() if k <= E else new(0, E, T, k)
        self.weights = torch.rand((T, k), generator=g, device=device) / 16
        self.weights.scatter_(1, new(0, k, T, 1), 1.0)

    def _hidden(self, which, at):
        """(T, k, n) sums of a first half's weight at columns `at` (T, k, n), in 64 bits."""
        b, s = self.w[which]
        T, k, n = at.shape
        out = 0.0
        for pos in ([self.p, torch.full_like(self.p, self.q)] if self.pairs else [self.p]):
            flat = (self.ids[:, :, None] * self.I + at).flatten()
            rows_b = b.flatten(0, 1)
            rows_s = s.flatten(0, 1)
            pos3 = pos[:, None, None].expand(T, k, n).flatten()
            byte = rows_b[flat, pos3 // 2].int()
            code = torch.where(pos3 % 2 == 1, byte >> 4, byte & 15).cpu()
            w = m4.VALUES[code.long()] * m4.scale_ref(rows_s[flat, pos3 // 32].cpu())
            xv = self.x.gather(1, pos[:, None]).double().cpu()[:, :, None].expand(T, k, n)
            out = out + w.view(T, k, n) * xv
        return out

    def result(self, out, held=lambda h: h):
        """y (T, D) in 64 bits and a bound of what 32 bits make of it; `held` is what becomes of h between the halves."""
        c = self.c[self.ids]  # (T, k, D): the column of h that counts
        b, s = self.w[2]
        byte = b[self.ids].gather(3, (c // 2)[..., None])[..., 0].int()
        code = torch.where(c % 2 == 1, byte >> 4, byte & 15).cpu()
        wd = m4.VALUES[code.long()] * m4.scale_ref(s[self.ids].gather(3, (c // 32)[..., None])[..., 0].cpu())
        wt = self.weights.double().cpu()[:, :, None]
        ks = self.ids.shape[1]
        h, amps = [], 0.0
        for at in ([c, c + 1] if self.pairs else [c]):
            a, _, amp = act_ref("silu", self._hidden(0, at))
            h.append(wt * a * self._hidden(1, at))
            amps = amp  # (the two have one gate)
        terms = [held(h[0]), -held(h[1])] if self.pairs else [held(h[0])]
        y = (wd * sum(terms)).sum(1)
        # Of the activation's 40 + 16 amp roundings (int8_util.gated_bound) all but those of u, its two products and
        # the weight are in both columns of a pair alike: they grow with the difference.  The first: u's 4, two products, the
        # second half's 3 parts and sums of 2 k + 8 terms, of each column's.
        of = sum(v.abs() for v in h)
        common = (h[0] - h[1]).abs() if self.pairs else h[0].abs()
        bound = (wd.abs() * (of * (14 + 2 * ks) + common * (40 + 16 * amps)) * U).sum(1)
        return y, bound + round_bound(y, out) + 2.0 ** -120
