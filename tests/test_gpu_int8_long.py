"""int8 x int8 operators over more rows and elements than one launch may have threads
(2^32), on rows of a few elements, and around the ends of the row ranges they are
launched in."""
import pytest
import torch

qmm = pytest.importorskip("gemv_only_quant_amd")
pytestmark = pytest.mark.gpu

RANGE = 1 << 22  # rows of one launch


def test_quantize_2_to_26_rows():
    """One element a row: the code is +-127 (0 of 0), the scale |x| / 127."""
    m = (1 << 26) + 5
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((m, 1), generator=g, device="cuda", dtype=torch.bfloat16)
    x[::1001] = 0
    q, s = qmm.quantize_tokens(x)
    assert torch.equal(s, (x[:, 0].double().abs() / 127).float())
    assert torch.equal(q[:, 0], (127 * torch.sign(x[:, 0].float())).to(torch.int8))


def test_empty_sums_of_2_to_24_rows():
    m = (1 << 24) + 3
    x = torch.empty((m, 0), dtype=torch.int8, device="cuda")
    w = torch.empty((1, 0), dtype=torch.int8, device="cuda")
    out = torch.full((m, 1), 7.0, device="cuda")
    one = torch.ones(m, device="cuda")
    qmm.w8a8_gemm(x, w, one[:1], sx=one, out=out)
    assert (out == 0).all()


def test_empty_gradient_of_2_to_32_elements():
    m, k = (1 << 21) - 300, 2100
    e = lambda *s, t=torch.int8: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    torch.full((m, k), 7.0, dtype=torch.bfloat16, device="cuda")  # what dx's memory holds before
    dx, _ = qmm.w8a8_gemm_backward(e(m, 0, t=torch.bfloat16), None, None, e(0, 2112)[:, :k],
                                   e(0, t=torch.float32), weight_grad=False)
    for i in range(0, m, 1 << 19):
        assert (dx[i:i + (1 << 19)] == 0).all()


@pytest.mark.parametrize("codes", [True, False])
def test_products_of_more_rows_than_a_launch(codes):
    """Values that are codes times a power of two (each row has a 127): the quantizer gives
    the codes back, whole sums stay below 2^24, and every result is exact."""
    m, k, n = RANGE + 70, 12, 3
    g = torch.Generator(device="cuda").manual_seed(2)
    c = torch.randint(-127, 128, (m, 16), generator=g, device="cuda", dtype=torch.int8)
    c[:, 5] = 127
    w = torch.randint(-128, 128, (n, 16), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.tensor([0.5, 1.0, 4.0], device="cuda")
    sx = 2.0 ** (torch.arange(m, device="cuda") % 7 - 3).float()
    left = dict(x=c[:, :k], sx=sx) if codes else dict(x=c[:, :k].float() * sx[:, None])
    sums = torch.stack([(c[:, :k].double() * w[j, :k].double()).sum(1) for j in range(n)], 1)
    want = (sums * (sx[:, None] * sw).double()).float()
    assert torch.equal(qmm.w8a8_gemm(W=w[:, :k], sw=sw, **left), want)
    # a gate of one in every row (its weight takes the 127 alone): silu has one value a row scale
    wg = torch.zeros((n, 16), dtype=torch.int8, device="cuda")
    wg[:, 5] = 1
    sg = torch.full((n,), 1 / 128, device="cuda")
    h = qmm.w8a8_gated(left["x"], wg[:, :k], sg, w[:, :k], sw, sx=left.get("sx"))
    gate = (127 * sx.double() / 128)[:, None]
    ref = gate * torch.sigmoid(gate) * want.double()
    # as the gated product's bound: 40 + 16 |g| units of 2^-24, |g| at most 8
    assert ((h.double() - ref).abs() <= ref.abs() * (40 + 16 * 8) * 2.0 ** -24).all()
