"""A gated feed-forward layer on int8 weights and activations: served, and trained.

    python examples/int8_feed_forward.py [--tokens 512] [--width 1024] [--hidden 2752] [--steps 20]

The layer is y = (act(x Wg^t) * (x Wu^t)) Wd^t.  Serving keeps the int8 weights with
a scale for each output channel and quantizes activations for each token: two
calls a layer, for one token as for a prompt.  Training keeps fp32 weights
beside them, quantizes them anew each step, and takes the gradients of the
dequantized weights for theirs (the straight-through estimate).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gemv_only_quant_amd as qmm  # noqa: E402


class FeedForward:
    def __init__(self, width, hidden, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        new = lambda n, k: torch.randn((n, k), generator=g, device=device) / k ** 0.5  # noqa: E731
        self.master = [new(hidden, width), new(hidden, width), new(width, hidden)]
        self.quantize()

    def quantize(self):
        """int8 weights from the fp32 ones: a weight's rows are quantized as
        tokens are, max |w| / 127 for each."""
        self.wg, self.wu, self.wd = (qmm.quantize_tokens(w) for w in self.master)

    def serve(self, x, act="silu"):
        h = qmm.w8a8_gated(x, *self.wg, *self.wu, act=act, out_dtype=x.dtype)
        return qmm.w8a8_gemm(h, *self.wd, out_dtype=x.dtype)

    def forward(self, x, act="silu"):
        """As serve, with what the gradients need: the codes and scales of both
        activations."""
        xq, sx = qmm.quantize_tokens(x)
        h = qmm.w8a8_gated(xq, *self.wg, *self.wu, act=act, sx=sx, out_dtype=x.dtype)
        hq, sh = qmm.quantize_tokens(h)
        y = qmm.w8a8_gemm(hq, *self.wd, sx=sh, out_dtype=x.dtype)
        return y, (xq, sx, hq, sh)

    def backward(self, dy, kept, act="silu"):
        """(dx, [dWg, dWu, dWd]) of dy's type."""
        xq, sx, hq, sh = kept
        dh, dwd = qmm.w8a8_gemm_backward(dy, hq, sh, *self.wd)
        dx, dwg, dwu = qmm.w8a8_gated_backward(dh, xq, sx, *self.wg, *self.wu, act=act)
        return dx, [dwg, dwu, dwd]

    def step(self, grads, rate):
        for w, g in zip(self.master, grads):
            w.add_(g.float(), alpha=-rate)
        self.quantize()


def train(tokens=512, width=1024, hidden=2752, steps=20, rate=0.05, log=print):
    """Fits a layer to another one's outputs; returns the losses."""
    teacher, student = FeedForward(width, hidden, seed=1), FeedForward(width, hidden, seed=2)
    g = torch.Generator(device="cuda").manual_seed(3)
    losses = []
    for i in range(steps):
        x = torch.randn((tokens, width), generator=g, device="cuda").bfloat16()
        target = teacher.serve(x)
        y, kept = student.forward(x)
        diff = y.float() - target.float()
        losses.append(float(diff.square().mean()))
        dx, grads = student.backward((diff * (2.0 / tokens)).bfloat16(), kept)
        student.step(grads, rate)
        log(f"step {i}: loss {losses[-1]:.5f}")
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=2752)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    layer = FeedForward(a.width, a.hidden)
    x = torch.randn((a.tokens, a.width), device="cuda").bfloat16()
    # one token at a time gives what the whole prompt gives, bit for bit: the
    # sums are whole numbers, and a token's scale is its own
    whole = layer.serve(x)
    alone = torch.cat([layer.serve(x[i:i + 1]) for i in range(3)])
    print("one token at a time equals the prompt:", bool(torch.equal(alone, whole[:3])))
    train(a.tokens, a.width, a.hidden, a.steps)


if __name__ == "__main__":
    main()
