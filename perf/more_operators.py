"""The operators on microscaled 4-bit floating point as a user's program calls
them, beside their plain form: what the cases are, how their inputs are made,
one pass, and what a pass cannot do without.

    quantize  x (M, K) -> codes and scales -> the values that they stand for
    gemm      y = x^ W^t                       (M, K) x (N, K) -> (M, N)
    moe       y[t] = sum_j w[t, j] Wd_e (act(Wg_e x[t]) * (Wu_e x[t])),  e = ids[t, j]

A row's 32 values of a block share the scale X = 2^(floor(log2 max |x|) - 2), held
as a byte e with X = 2^(e - 127); a value's 4 bits are x / X rounded to nearest
even among 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives, 6 where it is beyond.
x^ are the activations so quantized; the weights are in this format throughout.
The mixture of experts takes the activations as they are.  Its experts are the k
largest of a token's logits, weighted by the softmax over them or over all, or
are given with their weights; an index that names no expert counts for nothing.
"""
import math

import torch

own = False

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}


def listed():
    return [
        # one token's activations
        dict(name="quantize_1x4096_bf16", op="quantize", m=1, k=4096, x="bf16", out="bf16"),
        # odd rows, fp32
        dict(name="quantize_777x1001_fp32", op="quantize", m=777, k=1001, x="fp32", out="fp32"),
        # a layer's weights
        dict(name="quantize_11008x4096_bf16", op="quantize", m=11008, k=4096, x="bf16", out="bf16"),
        # one token through a square projection: latency
        dict(name="gemm_1x4096x4096_bf16", op="gemm", m=1, k=4096, n=4096, x="bf16", out="bf16"),
        # a small decode batch through a long, narrow projection
        dict(name="gemm_16x14336x1024_fp16", op="gemm", m=16, k=14336, n=1024, x="fp16", out="fp32"),
        # a decode batch of 64 through a wide projection
        dict(name="gemm_64x4096x14336_bf16", op="gemm", m=64, k=4096, n=14336, x="bf16", out="bf16"),
        # a ragged batch of prompts on odd widths
        dict(name="gemm_333x1001x2777_fp32", op="gemm", m=333, k=1001, n=2777, x="fp32", out="fp32"),
        # a long prompt
        dict(name="gemm_4096x4096x11008_bf16", op="gemm", m=4096, k=4096, n=11008, x="bf16", out="bf16"),
        # one token through a layer of many small experts
        dict(name="moe_1x2048x768_e128k8_bf16", op="moe", t=1, d=2048, i=768, e=128, k=8, x="bf16", out="bf16",
             act="silu", route="chosen"),
        # five tokens, odd widths, fp32, the router's own choice given (a third of it on other machines)
        dict(name="moe_5x1001x777_e16k4_fp32", op="moe", t=5, d=1001, i=777, e=16, k=4, x="fp32", out="fp32",
             act="gelu", route="ids"),
        # a decode batch through a few large experts
        dict(name="moe_16x4096x14336_e8k2_bf16", op="moe", t=16, d=4096, i=14336, e=8, k=2, x="bf16", out="bf16",
             act="silu", route="chosen"),
        # a larger batch through many small experts, weighted by the softmax over all
        dict(name="moe_64x2048x1408_e64k6_fp16", op="moe", t=64, d=2048, i=1408, e=64, k=6, x="fp16", out="fp16",
             act="gelu_tanh", route="all"),
    ]


LARGEST = 4096 * 4096 * 11008
MOST_WEIGHTS = 8 * 4096 * 14336


def draw(rng):
    """Rows from one token to a long prompt, widths from 64 to 14336, odd ones
    half of the time; mixtures of 2 to 128 experts for 1 to 64 tokens.  No more
    products, weights or values than the largest listed case of the operator."""
    op = rng.choice(["quantize", "gemm", "gemm", "moe", "moe"])

    def size(lo, hi):
        v = round(math.exp(rng.uniform(math.log(lo), math.log(hi))))
        return v if rng.random() < 0.5 or v < 32 else 32 * (v // 32)

    case = dict(op=op, x=rng.choice(["bf16", "fp16", "fp32"]), out=rng.choice(["bf16", "fp16", "fp32"]))
    if op == "moe":
        d, i = size(64, 4096), size(64, 14336)
        e = max(2, min(size(2, 128), MOST_WEIGHTS // (d * i)))
        case.update(t=rng.choice([1, 1, 2, 3, size(1, 64), size(1, 64)]), d=d, i=i, e=e,
                    k=rng.randint(1, min(8, e)), act=rng.choice(["silu", "gelu", "gelu_tanh"]),
                    route=rng.choice(["chosen", "all", "ids"]))
        return case
    case["k"] = k = size(64, 14336)
    if op == "quantize":
        case["m"] = max(1, min(size(1, 8192), 11008 * 4096 // k))
    else:
        case["n"] = n = size(64, 14336)
        case["m"] = max(1, min(size(1, 8192), LARGEST // (n * k)))
    return case


# ---------------------------------------------------------------- the format, plainly
def _quantize(x):
    """(codes, scale bytes) of x (M, K): one code per byte, rows of whole blocks.
    Quotients by powers of two are exact; the borders between codes decide them."""
    m, k = x.shape
    v = torch.zeros((m, -(-k // 32) * 32), dtype=torch.float64, device=x.device)
    v[:, :k] = x
    v = v.view(m, -1, 32)
    top = v.abs().amax(2)
    # floor(log2): frexp's exponent counts from [0.5, 1)
    e = (torch.frexp(top)[1] - 3).clamp(-127, 127)
    e = torch.where(top > 0, e, torch.full_like(e, -127))
    a = v.abs() / torch.exp2(e.double())[:, :, None]
    c = torch.zeros(v.shape, dtype=torch.uint8, device=x.device)
    for border, up in ((0.25, 0), (0.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5.0, 0)):
        c += (a >= border) if up else (a > border)
    c += 8 * torch.signbit(v)
    return c.view(m, -1), (e + 127).to(torch.uint8)


def _two_a_byte(c):
    """Codes in pairs, the first in the low half."""
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _values(codes, scales):
    """fp32 values of packed pairs of codes (..., K / 2) and scale bytes (..., K / 32)."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    v = table[c.int()].unflatten(-1, (-1, 32))
    return (v * torch.exp2(scales.float() - 127.0)[..., None]).flatten(-2)


# ---------------------------------------------------------------- inputs
def _activations(m, k, g):
    """Rows of unit variance with a few channels 16 times larger, as a
    transformer's residual stream has them."""
    x = torch.randn((m, k), generator=g, device="cuda")
    loud = torch.rand((k,), generator=g, device="cuda") < 0.002
    return x * (1.0 + 15.0 * loud)


def _weight(n, k, g):
    """(N, K / 2) pairs of codes and (N, K / 32) scale bytes of a normal weight
    whose products with unit rows have about unit variance."""
    w = torch.randn((n, -(-k // 32) * 32), generator=g, device="cuda") / math.sqrt(k)
    w[:, k:] = 0.0
    q, s = [], []
    for part in w.split(4096):  # the quantizer's 64-bit steps, some rows at a time
        c, e = _quantize(part)
        q.append(_two_a_byte(c))
        s.append(e)
    return torch.cat(q), torch.cat(s)


def _experts(count, n, k, g):
    """An expert each: the weights of a few, cut at another row for every one
    (64-bit steps on all of them would take longer than everything else)."""
    few = [_weight(n, k, g) for _ in range(min(count, 2))]
    q, s = [], []
    for e in range(count):
        cq, cs = few[e % len(few)]
        by = int(torch.randint(n, (1,), generator=torch.Generator().manual_seed(g.initial_seed() + e)))
        q.append(torch.roll(cq, by, 0))
        s.append(torch.roll(cs, by, 0))
    return torch.stack(q), torch.stack(s)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    state = dict(case=case)
    if case["op"] == "moe":
        t, d, i, e, k = (case[n] for n in ("t", "d", "i", "e", "k"))
        state["x"] = _activations(t, d, g).to(TYPES[case["x"]])
        state["w"] = [_experts(e, n, m, g) for n, m in ((i, d), (i, d), (d, i))]
        logits = 2.0 * torch.randn((t, e), generator=g, device="cuda")
        if case["route"] == "ids":
            # a router that has chosen already, and whose machine holds only some of the experts
            ids = torch.rand((t, e), generator=g, device="cuda").argsort(1)[:, :k]
            away = torch.rand((t, k), generator=g, device="cuda") < 1 / 3
            state["ids"] = torch.where(away, torch.full_like(ids, -1), ids).to(torch.int32)
            state["weights"] = torch.rand((t, k), generator=g, device="cuda") / k
        else:
            state["logits"] = logits
    else:
        state["x"] = _activations(case["m"], case["k"], g).to(TYPES[case["x"]])
        if case["op"] == "gemm":
            state["w"] = [_weight(case["n"], case["k"], g)]
    if own:
        import gemv_only_quant_amd as qmm

        # laid out once, as a model is loaded
        state["packed"] = [qmm.mx4_pack(q, s) for q, s in state.get("w", ())]
    return state


# ---------------------------------------------------------------- plain form
def _act(kind, g):
    if kind == "silu":
        return g / (1.0 + torch.exp(-g))
    if kind == "gelu":
        return g * 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _chosen(case, state):
    """(T, k) experts and weights."""
    if case["route"] == "ids":
        return state["ids"].long(), state["weights"]
    lg = state["logits"]
    top, ids = torch.sort(lg, dim=1, descending=True, stable=True)
    top, ids = top[:, :case["k"]], ids[:, :case["k"]]
    ex = torch.exp(top - top[:, :1])
    of = ex.sum(1, keepdim=True) if case["route"] == "chosen" else torch.exp(lg - top[:, :1]).sum(1, keepdim=True)
    return ids, ex / of


def _plain(state):
    case = state["case"]
    out = TYPES[case["out"]]
    if case["op"] != "moe":
        c, s = _quantize(state["x"])
        x = _values(_two_a_byte(c), s)
        if case["op"] == "quantize":
            return x[:, :case["k"]].to(out)
        return (x @ _values(*state["w"][0]).t()).to(out)
    d, i = case["d"], case["i"]
    x = state["x"].float()
    ids, weights = _chosen(case, state)
    (gq, gs), (uq, us), (dq, ds) = state["w"]
    y = torch.zeros_like(x)
    if ids.numel() <= case["e"]:
        # few choices: each one's own three weights
        for j in range(case["k"]):
            e = ids[:, j].clamp(min=0)
            w = weights[:, j] * (ids[:, j] >= 0)
            g = torch.matmul(_values(gq[e], gs[e])[:, :, :d], x[:, :, None])[:, :, 0]
            u = torch.matmul(_values(uq[e], us[e])[:, :, :d], x[:, :, None])[:, :, 0]
            h = _act(case["act"], g) * u
            y += w[:, None] * torch.matmul(_values(dq[e], ds[e])[:, :, :i], h[:, :, None])[:, :, 0]
    else:
        # many: every expert on all tokens, weighted by 0 where it is not theirs
        for e in range(case["e"]):
            w = (weights * (ids == e)).sum(1)
            g, u = x @ _values(gq[e], gs[e])[:, :d].t(), x @ _values(uq[e], us[e])[:, :d].t()
            h = _act(case["act"], g) * u
            y += w[:, None] * (h @ _values(dq[e], ds[e])[:, :i].t())
    return y.to(out)


# ---------------------------------------------------------------- the framework's calls
def _calls(state):
    import gemv_only_quant_amd as qmm

    case = state["case"]
    out = TYPES[case["out"]]
    if case["op"] == "quantize":
        q, s = qmm.mx4_quantize(state["x"])
        return qmm.mx4_dequantize(q, s, case["k"], out_dtype=out)
    if case["op"] == "gemm":
        return qmm.mx4_gemm(state["x"], state["packed"][0], case["n"], out_dtype=out)
    if case["route"] == "ids":
        route = dict(ids=state["ids"], weights=state["weights"])
    else:
        route = dict(logits=state["logits"], top_k=case["k"], renormalize=case["route"] == "chosen")
    return qmm.mx4_moe(state["x"], *state["packed"], case["i"], act=case["act"], out_dtype=out, **route)


def run(state):
    return _calls(state) if own else _plain(state)


def work(case):
    def coded(n, k):
        return n * (-(-k // 32)) * 17

    if case["op"] == "quantize":
        m, k = case["m"], case["k"]
        # values in, codes and scales out; those in, values out
        return {"bytes": m * k * (SIZE[case["x"]] + SIZE[case["out"]]) + 2 * coded(m, k), "flops": 2 * m * k}
    if case["op"] == "gemm":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": m * k * SIZE[case["x"]] + coded(n, k) + m * n * SIZE[case["out"]], "flops": 2 * m * n * k}
    t, d, i, e, k = (case[n] for n in ("t", "d", "i", "e", "k"))
    share = k / e * (2 / 3 if case["route"] == "ids" else 1)
    met = e * (1 - (1 - share) ** t)  # experts that some token chose, on average
    return {"bytes": round(met * (2 * coded(i, d) + coded(d, i))) + t * d * (SIZE[case["x"]] + SIZE[case["out"]]),
            "flops": round(6 * t * share * e * d * i)}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The definitions in 64 bits: a value's step is 2^-1 of its own power of two,
    from 1 up; halves go to the even multiple."""
    state = prepare(case, seed)

    def rounded(v):
        rows, cols = v.shape
        b = torch.nn.functional.pad(v.double(), (0, -cols % 32)).reshape(rows, -1, 32)
        top = b.abs().max(dim=-1, keepdim=True).values
        size = torch.where(top > 0, torch.floor(torch.log2(top)), torch.full_like(top, -127.0))
        # log2 rounds: a top next to a power of two may come out on its other side
        size = size + (torch.exp2(size + 1) <= top).double() - (torch.exp2(size) > top).double() * (top > 0)
        unit = torch.exp2((size - 2).clamp(-127, 127))
        r = b / unit
        step = torch.where(r.abs() >= 4, 2.0, torch.where(r.abs() >= 2, 1.0, 0.5)).double()
        return ((torch.round(r / step) * step).clamp(-6, 6) * unit).reshape(rows, -1)[:, :cols]

    def weight(q, s, cols):
        pair = torch.stack((q % 16, q // 16), dim=2).reshape(q.shape[0], -1).long()
        sign, exp, man = pair // 8, pair // 2 % 4, pair % 2
        size = torch.where(exp > 0, (1 + man / 2.0).double() * 2.0 ** (exp - 1).double(), man.double() / 2)
        unit = torch.ldexp(torch.ones_like(s, dtype=torch.float64), s.int() - 127)
        return ((1 - 2 * sign).double() * size * unit.repeat_interleave(32, dim=1))[:, :cols]

    if case["op"] == "quantize":
        return rounded(state["x"])
    if case["op"] == "gemm":
        return torch.mm(rounded(state["x"]), weight(*state["w"][0], case["k"]).t())
    x = state["x"].double()
    if "ids" in state:
        share = torch.zeros((case["t"], case["e"] + 1), dtype=torch.float64, device="cuda")
        share.scatter_add_(1, state["ids"].long() % (case["e"] + 1), state["weights"].double())  # -1: the last column
    else:
        p = torch.softmax(state["logits"].double(), 1)
        keep = torch.zeros_like(p)
        keep.scatter_(1, torch.topk(p, case["k"], dim=1).indices, 1.0)
        share = p * keep
        if case["route"] == "chosen":
            share = share / share.sum(1, keepdim=True)
    y = torch.zeros_like(x)
    (gq, gs), (uq, us), (dq, ds) = state["w"]
    for e in range(case["e"]):
        g, u = (torch.mm(x, weight(q[e], s[e], case["d"]).t()) for q, s in ((gq, gs), (uq, us)))
        if case["act"] == "gelu":
            p = 0.5 * torch.erfc(-g / math.sqrt(2.0))
        else:
            p = torch.sigmoid(g if case["act"] == "silu" else 2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g.pow(3)))
        y += share[:, e:e + 1] * torch.mm(g * p * u, weight(dq[e], ds[e], case["i"]).t())
    return y
