"""Microscaled 4-bit operators where offsets pass 32 bits: operands and results of more than 2^32 bytes, whose ends are
compared with calls on those alone."""
import pytest
import torch

import mx4_util as m4

pytestmark = pytest.mark.gpu
qmm = pytest.importorskip("gemv_only_quant_amd")


def free():
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def test_quantizer_of_many_values():
    M, K = (1 << 21) + 5, 2080  # 8.7 GB of values, 2.2 of codes
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    x.fill_(0.5)
    end = torch.randn((7, K), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    x[-7:] = end
    q, s = qmm.mx4_quantize(x)
    want = qmm.mx4_quantize(end)
    assert torch.equal(q[-7:], want[0]) and torch.equal(s[-7:], want[1])
    assert torch.equal(q[M // 2], q[0]) and torch.equal(s[M // 2], s[0])
    x.zero_()
    y = qmm.mx4_dequantize(q, s, K, out=x)
    assert torch.equal(y[-7:], qmm.mx4_dequantize(*want, K, out_dtype=torch.bfloat16)) and bool((y[M // 2] == 0.5).all())
    del x, y, q, s
    free()


@pytest.mark.parametrize("m", [1, 20, 100, 400])
def test_product_with_a_long_weight(m):
    N, K = 530000, 16000  # 4.6 GB of weight
    n = 48  # columns that are not zero: the last three strips
    bytes_ = qmm.mx4_packed_bytes(N, K)
    W = torch.zeros(bytes_, dtype=torch.uint8, device="cuda")
    q, s = m4.weight(n, K, 3)
    end = qmm.mx4_pack(q.cuda(), s.cuda())
    assert N % 16 == 0 and bytes_ > 1 << 32
    W[bytes_ - end.numel():] = end
    x = m4.tokens(m, K, 1, torch.bfloat16).cuda()
    y = qmm.mx4_gemm(x, W, N, out_dtype=torch.bfloat16)
    xv, wv = m4.values_ref(*m4.quantize_ref(x.cpu())), m4.values_ref(q, s)
    m4.assert_close(y[:, N - n:], xv @ wv.t(), m4.gemm_bound(xv, wv, torch.bfloat16), "end")
    assert bool((y[:, :N - n] == 0).all())
    del W, y
    free()


def test_product_of_many_results():
    M, N, K = 70000, 33000, 64  # 4.6 GB of y
    q, s = m4.weight(N, K, 2)
    W = qmm.mx4_pack(q.cuda(), s.cuda())
    x = torch.randn((M, K), device="cuda").bfloat16()
    y = qmm.mx4_gemm(x, W, N, out_dtype=torch.bfloat16)
    for i in (0, 32539, M - 300):  # (row 32540 starts about 2^31 bytes in)
        assert torch.equal(y[i:i + 300], qmm.mx4_gemm(x[i:i + 300].contiguous(), W, N, out_dtype=torch.bfloat16))
    del x, y
    free()


@pytest.mark.parametrize("T,k", [(1, 2), (5, 3), (12, 2), (64, 8)])
def test_mixture_of_many_experts(T, k):
    D, I, E, n = 2100, 3700, 1024, 2  # 4.7 to 5.2 GB for each of the three weights
    at = torch.tensor([700, 1023])
    packed, values = [], []
    for j, (rows, cols) in enumerate(((I, D), (I, D), (D, I))):
        qs = [m4.weight(rows, cols, 10 * j + i) for i in range(n)]
        some = qmm.mx4_pack(torch.stack([q for q, _ in qs]).cuda(), torch.stack([s for _, s in qs]).cuda())
        packed.append(torch.zeros((E, some.shape[1]), dtype=torch.uint8, device="cuda"))
        packed[-1][at.cuda()] = some
        values.append(torch.stack([m4.values_ref(q, s, cols) for q, s in qs]))
    assert packed[0].numel() > 1 << 32 and packed[2].numel() > 1 << 32
    g = torch.Generator().manual_seed(T)
    v, lg = m4.tokens(T, D, 1, torch.bfloat16), torch.randn((T, n), generator=g)
    full = torch.full((T, E), -float("inf"))
    full[:, at] = lg
    y = qmm.mx4_moe(v.cuda(), *packed, I, logits=full.cuda(), top_k=k, out_dtype=torch.bfloat16)
    ref, bound = m4.moe_ref("silu", v, *values, *m4.route_ref(lg, min(k, n), True), torch.bfloat16)
    m4.assert_close(y, ref, bound, f"experts {T}")
    del packed
    free()


@pytest.mark.parametrize("K", [(1 << 20) - 1, (1 << 20) - 31, (1 << 20) - 32])
def test_longest_rows(K):
    """K up to 2^20 - 1, through every call."""
    m, n = 2, 3
    q, s = m4.weight(n, K, 1)
    x = m4.tokens(m, K, 2, torch.bfloat16)
    W = qmm.mx4_pack(q.cuda(), s.cuda())
    assert W.numel() == qmm.mx4_packed_bytes(n, K)
    cq, cs = qmm.mx4_quantize(x.cuda())
    rq, rs = m4.quantize_ref(x)
    assert torch.equal(cq.cpu(), rq) and torch.equal(cs.cpu(), rs)
    xv, wv = m4.values_ref(rq, rs, K), m4.values_ref(q, s, K)
    assert torch.equal(qmm.mx4_dequantize(cq, cs, K).cpu().double(), xv)
    bound = m4.gemm_bound(xv, wv, torch.float32)
    m4.assert_close(qmm.mx4_gemm(cq, W, n, sx=cs), xv @ wv.t(), bound, "codes")
    m4.assert_close(qmm.mx4_gemm(x.cuda(), W, n), xv @ wv.t(), bound, "values")
