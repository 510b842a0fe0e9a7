"""The bounds of the mixtures of a term or two (mx4_terms) see an h of 16 bits or an x without its last part: planted in
the 64-bit reference, on the CPU."""
import pytest
import torch

import mx4_util as m4
from mx4_terms import Terms


def cut(v, bits):
    """v rounded to so many bits."""
    m, e = torch.frexp(v)
    return torch.ldexp((m * 2.0 ** bits).round() / 2.0 ** bits, e)


# T, D, I, E, k
SHAPES = [(1, 64, 64, 4, 2), (5, 100, 77, 6, 3), (64, 460, 330, 20, 8), (16, 300, 1000, 10, 8)]


@pytest.mark.parametrize("T,D,I,E,k", SHAPES)
@pytest.mark.parametrize("out", m4.TYPES)
@pytest.mark.parametrize("pairs", [False, True])
def test_bound_sees_a_short_hidden(T, D, I, E, k, out, pairs):
    """With the difference of a pair also where y itself has few bits."""
    t = Terms(T, D, I, E, k, torch.float32, pairs, 3, "cpu")
    y, bound = t.result(m4.TYPES[out])
    short = t.result(m4.TYPES[out], lambda h: cut(h, 16))[0]
    exact = t.result(m4.TYPES[out], lambda h: cut(h, 24))[0]
    assert ((exact - y).abs() <= bound).all()
    if pairs or out == "fp32":
        assert ((short - y).abs() > bound).any()


@pytest.mark.parametrize("T,D,I,E,k", SHAPES)
@pytest.mark.parametrize("x,bits", [("fp32", 16), ("fp16", 8)])
def test_bound_sees_a_short_x(T, D, I, E, k, x, bits):
    t = Terms(T, D, I, E, k, m4.TYPES[x], False, 4, "cpu")
    y, bound = t.result(torch.float32)
    t.x = cut(t.x.double(), bits)
    assert ((t.result(torch.float32)[0] - y).abs() > bound).any()
