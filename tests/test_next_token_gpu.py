"""The next-token example: its gradients against the formula in 64 bits and against differences, the operators run
together as it uses them, repeated to the bit and captured."""

import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import decoupled_momentum_optimizer_gb300 as dm
import train_next_token as ex
from model_ref import f64, norm_grad, norm_rstd

pytestmark = pytest.mark.gpu

V, D, FF, L, T = 150, 96, 160, 2, 300


def setup(seed=3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    model = ex.NextToken(V, D, FF, L)
    theta = model.init(gen)
    for i in range(L):
        model.part(theta, f"norm{i}").add_(torch.randn(D, generator=gen, device="cuda") * 0.1)
    model.quantize(theta)
    tokens = torch.randint(V, (T,), generator=gen, device="cuda")
    tokens[5::7] = 3  # a token that is named often
    return model, theta, tokens, torch.randint(V, (T,), generator=gen, device="cuda")


def exact(model, theta, tokens, targets):
    """(loss, logits, gradients by name) without any quantization, in 64 bits."""
    p = {name: model.part(theta, name).copy() for name in model.at}
    s, kept = p["embed"][tokens] * np.sqrt(D), []
    for i in range(L):
        r = norm_rstd(s, 1e-6)
        n = s * r[:, None] * p[f"norm{i}"]
        h = n @ p[f"w1.{i}"].T
        kept.append((s, r, n, h))
        s = s + np.maximum(h, 0) @ p[f"w2.{i}"].T
    r = norm_rstd(s, 1e-6)
    n = s * r[:, None] * p["norm"]
    logits = n @ p["embed"].T
    e = np.exp(logits - logits.max(1, keepdims=True))
    prob = e / e.sum(1, keepdims=True)
    rows = np.arange(len(tokens))
    loss = -np.log(prob[rows, targets]).mean()
    dl = prob.copy()
    dl[rows, targets] -= 1
    dl /= len(tokens)
    g = {"embed": dl.T @ n}
    ds, g["norm"], _, _ = norm_grad(dl @ p["embed"], s, p["norm"], r)
    for i in reversed(range(L)):
        s, r, n, h = kept[i]
        dh = (ds @ p[f"w2.{i}"]) * (h > 0)
        g[f"w2.{i}"], g[f"w1.{i}"] = ds.T @ np.maximum(h, 0), dh.T @ n
        ds, g[f"norm{i}"], _, _ = norm_grad(dh @ p[f"w1.{i}"], s, p[f"norm{i}"], r, ds)
    np.add.at(g["embed"], tokens, ds * np.sqrt(D))
    return loss, logits, g


def test_gradients_follow_the_formula():
    """Against unquantized 64-bit gradients.  e4m3 rounds an element by at most 2^-4 of it, 0.036 root mean square
    at worst, e5m2 by 0.072; a product's relative error is the root of the sum of its operands' squares.  Forward,
    a layer leaves 0.072 and the logits 0.09; backward, each of the two layers passes three operands in e5m2 and
    three in e4m3 on, from 0.08 behind the logits to 0.14 behind the last layer and 0.19 behind the first: below
    a quarter of each gradient's norm, a cosine above 0.968."""
    model, theta, tokens, targets = setup()
    logits, state = model.forward(tokens)
    loss, dlogits = ex.loss_and_gradient(logits, targets)
    grad = torch.zeros_like(theta)
    model.backward(dlogits, state, grad)
    want_loss, want_logits, want = exact(model, f64(theta), tokens.cpu().numpy(), targets.cpu().numpy())
    assert np.linalg.norm(f64(logits) - want_logits) <= 0.25 * np.linalg.norm(want_logits)
    assert np.isfinite(f64(grad)).all()
    for name, w in want.items():
        got = f64(model.part(grad, name))
        assert np.linalg.norm(got - w) <= 0.25 * np.linalg.norm(w), name
        assert (got * w).sum() >= 0.968 * np.linalg.norm(got) * np.linalg.norm(w), name


def test_formula_against_differences():
    model, theta, tokens, targets = setup()
    th, x, y = f64(theta), tokens.cpu().numpy(), targets.cpu().numpy()
    _, _, want = exact(model, th, x, y)
    rng = np.random.default_rng(0)
    for name, (start, shape) in model.at.items():
        for i in rng.integers(0, int(np.prod(shape)), 3):
            h = 1e-6
            up, down = th.copy(), th.copy()
            up[start + i] += h
            down[start + i] -= h
            diff = (exact(model, up, x, y)[0] - exact(model, down, x, y)[0]) / (2 * h)
            assert abs(diff - want[name].ravel()[i]) <= 1e-5 * np.abs(want[name]).max(), name


def run_step(model, theta, tokens, targets, grad):
    logits, state = model.forward(tokens)
    _, dlogits = ex.loss_and_gradient(logits, targets)
    model.backward(dlogits, state, grad)
    return dm.clip_grads(grad, 0.1)


def test_a_step_repeats_to_the_bit_and_from_a_graph():
    model, theta, tokens, targets = setup()
    out = []
    for _ in range(2):
        grad = torch.zeros_like(theta)
        out.append((run_step(model, theta, tokens, targets, grad), grad))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    norm, grad = out[0]
    assert abs(float(dm.grad_norm(grad)) - 0.1) <= 1e-6 and float(norm) > 0.1
    x, captured = tokens.clone(), torch.zeros_like(theta)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n = run_step(model, theta, x, targets, captured)
    for shift in (0, 1):
        x.copy_((tokens + shift) % V)
        graph.replay()
        want = torch.zeros_like(theta)
        assert torch.equal(n, run_step(model, theta, x, targets, want)) and torch.equal(captured, want)


def test_serving_agrees_with_the_forward_pass():
    """The few-token form rounds the norm's result to bfloat16 before its codes: logits apart by a few of bfloat16's
    steps, and the same token wherever the two likeliest are further apart."""
    model, theta, tokens, _ = setup()
    logits, _ = model.forward(tokens[:9])
    top = f64(logits.topk(2).values)
    clear = top[:, 0] - top[:, 1] > 0.1 * np.abs(f64(logits)).max()
    assert clear.any() and np.array_equal(f64(model.predict(tokens[:9]))[clear], f64(logits.argmax(-1))[clear])


def test_the_whole_loop_runs():
    losses, norms = ex.train(vocab=200, d=128, ff=256, tokens=256, steps=5, log=None)
    assert np.isfinite(losses).all() and np.isfinite(norms).all() and len(losses) == 10
    assert dm.device_fault() == 0
