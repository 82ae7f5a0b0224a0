"""Train a next-token model with every part of the package: tied embedding, norms, 8-bit products, clipping, the step.

    python examples/train_next_token.py --steps 30

    s_0 = E[token] sqrt(d),   s_{l+1} = s_l + relu(norm_l(s_l) W1_l^T) W2_l^T,   logits = norm(s_L) E^T

E [vocab, d], the norms' weights and W1 [ff, d], W2 [d, ff] of each layer live in one flat float32 shard theta, every
one at a multiple of 32 elements.  A step quantizes the matrices to 8 bits once; each of R replicas then runs its
batch: rows of E by token, norms that add the residual and leave 8-bit codes for the products, the products,
and the way back, every gradient written into the replica's flat float32 gradient (E's twice: by the output layer,
then the rows of the tokens added).  The gradient is clipped to a norm, and the decoupled-momentum step updates
theta from the replicas' gradients.  Nothing on the way waits for the device.
"""

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import decoupled_momentum_optimizer_gb300 as dm  # noqa: E402


class NextToken:
    """The model on a flat shard; gradients are written, not accumulated."""

    def __init__(self, vocab, d, ff, layers):
        self.vocab, self.d, self.ff, self.layers = vocab, d, ff, layers
        self.at, self.size = {}, 0
        shapes = [("embed", (vocab, d))]
        for i in range(layers):
            shapes += [(f"norm{i}", (d,)), (f"w1.{i}", (ff, d)), (f"w2.{i}", (d, ff))]
        for name, shape in shapes + [("norm", (d,))]:
            self.at[name] = (self.size, shape)
            self.size += (math.prod(shape) + 31) // 32 * 32

    def part(self, flat, name):
        """A parameter, or its gradient, as a slice of the flat shard."""
        start, shape = self.at[name]
        return flat[start:start + math.prod(shape)].reshape(shape)

    def init(self, gen):
        theta = torch.zeros(self.size, device="cuda")
        for name, (_, shape) in self.at.items():
            if name.startswith("norm"):
                self.part(theta, name).fill_(1.0)
            else:
                self.part(theta, name).normal_(0.0, shape[-1] ** -0.5, generator=gen)
        return theta

    def quantize(self, theta):
        """Once a step: every matrix by rows (forward) and by columns (input gradient)."""
        self.theta = theta
        self.q = {name: dm.fp8_quantize(self.part(theta, name), form="both", scales="tiles")
                  for name in self.at if not name.startswith("norm")}

    def forward(self, tokens):
        """float32 logits and what backward needs."""
        s = dm.embedding(tokens, self.part(self.theta, "embed"), scale=self.d ** 0.5, dtype=torch.bfloat16)
        z, saved = None, []
        for i in range(self.layers):
            n = dm.rms_norm(s, self.part(self.theta, f"norm{i}"), residual=z, values=False, form="both", save=True)
            h = dm.fp8_matmul(n.quantized[0], self.q[f"w1.{i}"][0])
            aq, at = dm.fp8_quantize(h, form="both", relu=True)
            s, z = n.total, dm.fp8_matmul(aq, self.q[f"w2.{i}"][0])
            saved.append((n, h, at))
        n = dm.rms_norm(s, self.part(self.theta, "norm"), residual=z, values=False, form="both", save=True)
        return dm.fp8_matmul(n.quantized[0], self.q["embed"][0], dtype=torch.float32), (tokens, saved, n)

    def backward(self, dlogits, state, grad):
        """Writes every gradient into the flat `grad`."""
        tokens, saved, n = state
        dl, dlt = dm.fp8_quantize(dlogits, fmt="e5m2", form="both")
        dm.fp8_matmul(dlt, n.quantized[1], out=self.part(grad, "embed"))
        ds, _ = dm.rms_norm_grad(dm.fp8_matmul(dl, self.q["embed"][1]), n.total, self.part(self.theta, "norm"), n.rstd,
                                 dweight=self.part(grad, "norm"))
        for i in reversed(range(self.layers)):
            n, h, at = saved[i]
            dz, dzt = dm.fp8_quantize(ds, fmt="e5m2", form="both")
            dm.fp8_matmul(dzt, at, out=self.part(grad, f"w2.{i}"))
            dh, dht = dm.fp8_quantize(dm.fp8_matmul(dz, self.q[f"w2.{i}"][1]), fmt="e5m2", form="both", gate=h)
            dm.fp8_matmul(dht, n.quantized[1], out=self.part(grad, f"w1.{i}"))
            ds, _ = dm.rms_norm_grad(dm.fp8_matmul(dh, self.q[f"w1.{i}"][1]), n.total, self.part(self.theta, f"norm{i}"),
                                     n.rstd, past=ds, dweight=self.part(grad, f"norm{i}"))
        dm.embedding_grad(tokens, ds, out=self.part(grad, "embed"), scale=self.d ** 0.5, add=True)

    def predict(self, tokens):
        """The likeliest next tokens of a few: the form that serves them."""
        s = dm.embedding(tokens, self.part(self.theta, "embed"), scale=self.d ** 0.5, dtype=torch.bfloat16)
        z = None
        for i in range(self.layers):
            n = dm.rms_norm(s, self.part(self.theta, f"norm{i}"), residual=z)
            s, z = n.total, dm.fp8_linear(dm.fp8_linear(n.out, self.q[f"w1.{i}"][0]).relu_(), self.q[f"w2.{i}"][0])
        n = dm.rms_norm(s, self.part(self.theta, "norm"), residual=z)
        return dm.fp8_linear(n.out, self.q["embed"][0], dtype=torch.float32).argmax(-1)


def loss_and_gradient(logits, targets):
    """Mean cross-entropy, a device scalar, and its gradient by the logits (float32)."""
    logp = logits.log_softmax(-1)
    loss = -logp.gather(1, targets[:, None]).mean()
    dlogits = logp.exp_()
    dlogits.scatter_add_(1, targets[:, None], torch.full_like(targets[:, None], -1, dtype=torch.float32))
    return loss, dlogits / len(targets)


def train(vocab=500, d=256, ff=512, layers=2, tokens=1024, replicas=2, steps=30, max_norm=1.0, k=4, lr=2e-3, beta=0.9, seed=0,
          log=print):
    """Learns a random successor for each token; returns (losses, gradient norms), one of each per step."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    model = NextToken(vocab, d, ff, layers)
    theta = model.init(gen)
    successor = torch.randperm(vocab, generator=gen, device="cuda")
    gs = [torch.zeros(model.size, device="cuda") for _ in range(replicas)]  # the padding stays zero
    ms = [torch.zeros(model.size, device="cuda") for _ in range(replicas)]
    losses, norms = [], []
    for step in range(steps):
        model.quantize(theta)
        for r in range(replicas):
            x = torch.randint(vocab, (tokens,), generator=gen, device="cuda")
            logits, state = model.forward(x)
            loss, dlogits = loss_and_gradient(logits, successor[x])
            model.backward(dlogits, state, gs[r])
            norms.append(dm.clip_grads(gs[r], max_norm))
            losses.append(loss)
        dm.step(theta, gs, ms, k=k, beta=beta, lr=lr, mode="demo", sign=True, seed=seed, step=step)
        if log and (step % 10 == 0 or step == steps - 1):
            log(f"step {step}: loss {losses[-1].item():.4f}, gradient norm {norms[-1].item():.3f}")
    return [v.item() for v in losses], [v.item() for v in norms]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--replicas", type=int, default=2)
    ap.add_argument("--max-norm", type=float, default=1.0)
    a = ap.parse_args()
    train(steps=a.steps, tokens=a.tokens, replicas=a.replicas, max_norm=a.max_norm)
