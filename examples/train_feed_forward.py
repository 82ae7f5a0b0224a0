"""Train a residual feed-forward layer with every part of the package.

    python examples/train_feed_forward.py --steps 30

    h = x W1^T,   y = x + dropout(dropout(relu(h)) W2^T),   loss = mean((y - target)^2)

W1 [ff, d] and W2 [d, ff] live in one flat float32 shard theta.  Every step quantizes them to 8 bits
once (both directions of the product share the values), then each of R replicas runs its own batch:
the products in 8 bits with a scale for each block of 128, relu and dropout applied while the hidden
activations are quantized, the weight gradients written straight into the replica's flat float32
gradient.  The decoupled-momentum step then updates theta from the replicas' gradients.  The dropout
masks are functions of (seed, step, site), so a step can be repeated exactly from theta, the momenta,
the seed and the step counter.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import decoupled_momentum_optimizer_gb300 as dm  # noqa: E402

HIDDEN, OUTPUT = 0, 1  # dropout sites


class FeedForward:
    """The layer on a flat shard; gradients are written, not accumulated."""

    def __init__(self, theta, d, ff, p):
        self.d, self.ff, self.p = d, ff, p
        self.w1, self.w2 = theta[:ff * d].view(ff, d), theta[ff * d:].view(d, ff)

    def quantize_weights(self):
        """Once a step: W1 and W2 by rows (forward) and by columns (input gradient)."""
        self.q1, self.q1t = dm.fp8_quantize(self.w1, form="both", scales="tiles")
        self.q2, self.q2t = dm.fp8_quantize(self.w2, form="both", scales="tiles")

    def forward(self, x, seed, step):
        """y and what backward needs; x is [tokens, d] in bfloat16."""
        xq, xt = dm.fp8_quantize(x, form="both")
        h = dm.fp8_matmul(xq, self.q1)
        aq, at = dm.fp8_quantize(h, form="both", relu=True, p=self.p, seed=seed, step=step, site=HIDDEN)
        z = dm.fp8_matmul(aq, self.q2)
        y = dm.dropout(z, self.p, seed=seed, step=step, site=OUTPUT, residual=x)
        return y, (xt, h, at)

    def backward(self, dy, saved, grad, seed, step):
        """Writes dW1 and dW2 into the flat `grad`; returns dx."""
        xt, h, at = saved
        g1, g2 = grad[:self.ff * self.d].view(self.ff, self.d), grad[self.ff * self.d:].view(self.d, self.ff)
        dz, dzt = dm.fp8_quantize(dy, fmt="e5m2", form="both", p=self.p, seed=seed, step=step, site=OUTPUT)
        dm.fp8_matmul(dzt, at, out=g2)
        da = dm.fp8_matmul(dz, self.q2t)
        dh, dht = dm.fp8_quantize(da, fmt="e5m2", form="both", gate=h, p=self.p, seed=seed, step=step, site=HIDDEN)
        dm.fp8_matmul(dht, xt, out=g1)
        return dy + dm.fp8_matmul(dh, self.q1t)

    def decode(self, x):
        """The layer on a few tokens without dropout."""
        return x + dm.fp8_linear(dm.fp8_linear(x, self.q1).relu_(), self.q2)


def train(d=768, ff=2048, tokens=1024, replicas=2, steps=30, p=0.1, k=4, lr=2e-4, beta=0.9, seed=0, log=print):
    """Fits the layer to a random one; returns the losses (one per step)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = 2 * d * ff
    theta = torch.randn(n, generator=gen, device="cuda") * 0.02
    teacher = torch.randn(n, generator=gen, device="cuda") * 0.02
    layer = FeedForward(theta, d, ff, p)
    gs = [torch.empty(n, device="cuda") for _ in range(replicas)]
    ms = [torch.zeros(n, device="cuda") for _ in range(replicas)]
    losses = []
    for step in range(steps):
        layer.quantize_weights()
        total = torch.zeros((), device="cuda")
        for r in range(replicas):
            x = torch.randn(tokens, d, generator=gen, device="cuda").bfloat16()
            t1, t2 = teacher[:ff * d].view(ff, d).bfloat16(), teacher[ff * d:].view(d, ff).bfloat16()
            target = x + (x @ t1.t()).relu_() @ t2.t()
            y, saved = layer.forward(x, seed + r, step)
            err = y - target
            total += err.float().square().mean() / replicas
            layer.backward(err * (2.0 / tokens), saved, gs[r], seed + r, step)
        dm.step(theta, gs, ms, k=k, beta=beta, lr=lr, mode="demo", sign=True, seed=seed, step=step)
        losses.append(total)
        if log and (step % 10 == 0 or step == steps - 1):
            log(f"step {step}: loss {losses[-1].item():.4f}")
    return [loss.item() for loss in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--replicas", type=int, default=2)
    ap.add_argument("--p", type=float, default=0.1)
    a = ap.parse_args()
    train(steps=a.steps, tokens=a.tokens, replicas=a.replicas, p=a.p)
