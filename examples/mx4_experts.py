"""A mixture-of-experts layer and an output projection on microscaled 4-bit weights, served.

    python examples/mx4_experts.py [--width 2048] [--hidden 768] [--experts 64] [--top-k 8] [--vocab 32000]

A step takes a few tokens (a decode batch) through router, experts and projection, and is captured once into
a graph and replayed; a prompt goes through the projection alone, in tiles.  Experts' weights are quantized and
laid out once; activations of the mixture stay as they are, the projection's are quantized by its call.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gemv_only_quant_amd as qmm  # noqa: E402


def laid_out(weights):
    """(E, N, K) or (N, K) values -> the layout that the products read."""
    n, k = weights.shape[-2:]
    codes, scales = qmm.mx4_quantize(weights.reshape(-1, k))
    shape = weights.shape[:-1]
    return qmm.mx4_pack(codes.view(*shape, -1), scales.contiguous().view(*shape, -1))


class Experts:
    def __init__(self, width, hidden, experts, top_k, vocab, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        new = lambda *s: torch.randn(s, generator=g, device=device) / s[-1] ** 0.5  # noqa: E731
        self.hidden, self.top_k, self.vocab = hidden, top_k, vocab
        self.router = new(experts, width)
        self.gate, self.up = laid_out(new(experts, hidden, width)), laid_out(new(experts, hidden, width))
        self.down, self.head = laid_out(new(experts, width, hidden)), laid_out(new(vocab, width))

    def layer(self, x):
        """x (T, width), up to 64 tokens -> x + the mixture of their experts."""
        logits = x.float() @ self.router.t()
        return x + qmm.mx4_moe(x, self.gate, self.up, self.down, self.hidden, logits=logits, top_k=self.top_k,
                               out_dtype=x.dtype)

    def project(self, x):
        """x (M, width), any M -> (M, vocab) fp32."""
        return qmm.mx4_gemm(x, self.head, self.vocab)

    def step(self, x):
        return self.project(self.layer(x))


def captured(fn, x):
    """A call that replays fn on what it copies into x's place."""
    at = x.clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        fn(at)  # (first calls set libraries up, which a capture must not see)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = fn(at)

    def call(x):
        at.copy_(x)
        graph.replay()
        return y

    return call


def main(argv=None, log=print):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=768)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--top-k", type=int, default=8)
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--tokens", type=int, default=4)
    a = ap.parse_args(argv)
    model = Experts(a.width, a.hidden, a.experts, a.top_k, a.vocab)
    x = [torch.randn((a.tokens, a.width), device="cuda").bfloat16() for _ in range(3)]
    replay = captured(model.step, x[0])
    same = [bool(torch.equal(replay(v), model.step(v))) for v in x]
    log(f"replayed steps equal eager ones: {same}")
    prompt = torch.randn((500, a.width), device="cuda").bfloat16()
    log(f"prompt: {tuple(model.project(prompt).shape)}")
    return same


if __name__ == "__main__":
    main()
