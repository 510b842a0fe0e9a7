"""The mixture's forms on sums of a term or two, within a few roundings whatever the sizes (mx4_terms); and what is not
finite in a row stays there, in each of them."""
import math

import pytest
import torch

import mx4_util as m4
from mx4_terms import Terms
from mx4_util import TYPES

qmm = pytest.importorskip("gemv_only_quant_amd")
pytestmark = pytest.mark.gpu

# (T, D, I, E, top_k) by the forms of the halves: few tokens in both; in the first alone; rows through LDS, their sums joined
# by the last workgroup and by a launch; an expert's rows held by one or two groups in the first, the second, both; in ranges
FORMS = [(1, 64, 64, 4, 2), (4, 72, 96, 40, 2), (4, 1032, 700, 40, 8), (4, 40, 2600, 20, 5), (5, 100, 77, 6, 3), (8, 700, 515, 5, 1),
         (16, 256, 128, 8, 2), (33, 96, 1040, 4, 4), (64, 130, 330, 300, 8), (64, 460, 40, 300, 8), (64, 460, 330, 260, 8),
         (16, 460, 330, 256, 32), (8, 460, 330, 256, 32), (5, 460, 330, 300, 32), (4, 897, 650, 128, 32),
         (64, 2100, 330, 260, 8), (64, 460, 2100, 260, 8), (20, 4000, 330, 300, 32), (16, 900, 9000, 40, 8),
         # few tokens whose h fits LDS in two turns, of as many chunks and of one less; three groups and ranges
         (3, 520, 768, 40, 8), (1, 72, 14336, 4, 2), (1, 72, 13500, 4, 2), (32, 900, 5000, 24, 8)]


def run(t, out):
    packed = [qmm.mx4_pack(q, s) for q, s in t.w]
    return qmm.mx4_moe(t.x, *packed, t.I, ids=t.ids, weights=t.weights, out_dtype=out)


@pytest.mark.parametrize("T,D,I,E,k", FORMS)
@pytest.mark.parametrize("x", TYPES)
def test_one_term(T, D, I, E, k, x):
    """Every bit of x, and of h."""
    t = Terms(T, D, I, E, k, TYPES[x], False, T + D, "cuda")
    y, bound = t.result(torch.float32)
    m4.assert_close(run(t, torch.float32), y, bound, f"{T} {D} {I} {E} {k}")


@pytest.mark.parametrize("T,D,I,E,k", FORMS)
@pytest.mark.parametrize("x,out", [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "bf16"), ("bf16", "fp32")])
def test_difference_of_two_terms(T, D, I, E, k, x, out):
    """Of nearly equal values of h: their last bits, whatever y's type."""
    t = Terms(T, D, I, E, k, TYPES[x], True, T + I, "cuda")
    y, bound = t.result(TYPES[out])
    m4.assert_close(run(t, TYPES[out]), y, bound, f"{T} {D} {I} {E} {k}")


@pytest.mark.parametrize("T,D,I,E,k", FORMS)
def test_not_finite_stays_in_its_row(T, D, I, E, k):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    byte = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device="cuda").to(torch.uint8)  # noqa: E731
    packed = [qmm.mx4_pack(byte(0, 256, E, n, 16 * m4.blocks(m)), byte(115, 120, E, n, m4.blocks(m)))
              for n, m in ((I, D), (I, D), (D, I))]
    lg = torch.randn((T, E), generator=g, device="cuda")
    for t in TYPES.values():
        x = torch.randn((T, D), generator=g, device="cuda").to(t)
        call = lambda v: qmm.mx4_moe(v, *packed, I, logits=lg, top_k=k)  # noqa: E731
        clean = call(x)
        assert torch.isfinite(clean).all()
        for row, at, bad in ((T - 1, D - 1, math.nan), (T // 2, 0, math.inf), (0, D // 2, -math.inf)):
            b = x.clone()
            b[row, at] = bad
            y = call(b)
            assert torch.isnan(y[row]).all(), (row, bad)
            y[row] = clean[row]
            assert torch.equal(y, clean), (row, bad)
