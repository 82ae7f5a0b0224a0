"""The feed-forward example: its gradients against the formula in 64 bits and against differences,
and the whole loop (quantize, products, dropout, decoupled-momentum step) from end to end."""

import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import decoupled_momentum_optimizer_gb300 as dm
import train_feed_forward as ex
import train_ref as ref

pytestmark = pytest.mark.gpu

D, FF, T = 96, 160, 130


def f64(t):
    return t.double().cpu().numpy()


def setup(p):
    gen = torch.Generator(device="cuda").manual_seed(3)
    theta = torch.randn(2 * D * FF, generator=gen, device="cuda") * 0.1
    x = torch.randn(T, D, generator=gen, device="cuda").bfloat16()
    dy = (torch.randn(T, D, generator=gen, device="cuda") * 1e-2).bfloat16()
    layer = ex.FeedForward(theta, D, FF, p)
    layer.quantize_weights()
    return theta, x, dy, layer


def exact(theta, x, p, dy):
    """(y, gradients, dx) of the layer without any quantization, in 64 bits."""
    w1, w2 = theta[:FF * D].reshape(FF, D), theta[FF * D:].reshape(D, FF)
    s = ref.drop_scale(p)
    k1, k2 = ref.keep_mask(T, FF, p, 7, 5, ex.HIDDEN), ref.keep_mask(T, D, p, 7, 5, ex.OUTPUT)
    h = x @ w1.T
    a = np.where(k1, np.maximum(h, 0) * s, 0)
    y = x + np.where(k2, (a @ w2.T) * s, 0)
    dz = np.where(k2, dy * s, 0)
    dh = np.where(k1 & (h > 0), (dz @ w2) * s, 0)
    return y, np.concatenate([(dh.T @ x).ravel(), (dz.T @ a).ravel()]), dy + dh @ w1


def cosine(a, b):
    return float((a * b).sum() / np.sqrt((a * a).sum() * (b * b).sum()))


@pytest.mark.parametrize("p", [0.0, 0.25])
def test_gradients_follow_the_formula(p):
    """Against unquantized 64-bit gradients: e4m3 rounds an element by at most 2^-4 of it and e5m2 by
    2^-3 (uniformly spread: 2^-4 / sqrt(3) and 2^-3 / sqrt(3), 0.04 and 0.07, root mean square at
    worst); through the chain of three products that is below 0.15 of the gradient's norm, a cosine
    above 0.985."""
    theta, x, dy, layer = setup(p)
    y, saved = layer.forward(x, 7, 5)
    grad = torch.full_like(theta, float("nan"))
    dx = layer.backward(dy, saved, grad, 7, 5)
    want_y, want_g, want_dx = exact(f64(theta), f64(x), p, f64(dy))
    assert np.isfinite(f64(grad)).all()
    for got, want in ((f64(y), want_y), (f64(grad), want_g), (f64(dx), want_dx)):
        assert np.linalg.norm(got - want) <= 0.15 * np.linalg.norm(want)
        assert cosine(got, want) > 0.985


def test_weight_gradients_are_the_products_of_their_operands():
    """Exactly what the quantized operands say, up to the products' own bound."""
    theta, x, dy, layer = setup(0.25)
    y, (xt, h, at) = layer.forward(x, 7, 5)
    grad = torch.empty_like(theta)
    layer.backward(dy, (xt, h, at), grad, 7, 5)
    dzt = dm.fp8_quantize(dy, fmt="e5m2", form="cols", p=0.25, seed=7, step=5, site=ex.OUTPUT)
    want, total = ref.product(f64(dzt.dequantize()), f64(at.dequantize()))
    got = f64(grad[FF * D:]).reshape(D, FF)
    assert (np.abs(got - want) <= ref.product_tolerance(total, T) + 2.0 ** -24 * np.abs(want)).all()


def test_gradient_against_differences():
    """The formula's gradient (checked against the kernels' above) against central differences of the
    64-bit loss sum(dy * y), where no hidden unit changes sign over the step."""
    theta, x, dy, _ = setup(0.25)
    th, xx, g = f64(theta), f64(x), f64(dy)
    _, want, _ = exact(th, xx, 0.25, g)
    for i in np.random.default_rng(0).integers(0, th.size, 20):
        eps = 1e-7
        up, down = th.copy(), th.copy()
        up[i] += eps
        down[i] -= eps
        diff = ((exact(up, xx, 0.25, g)[0] - exact(down, xx, 0.25, g)[0]) * g).sum() / (2 * eps)
        assert abs(diff - want[i]) <= 1e-6 * np.abs(want).max()


def test_decode_is_forward_without_dropout():
    theta, x, dy, layer = setup(0.0)
    y, _ = layer.forward(x, 0, 0)
    few = layer.decode(x[:3])
    # the hidden activations pass through bfloat16 either way; codes may round apart at that precision
    assert np.linalg.norm(f64(few) - f64(y[:3])) <= 0.02 * np.linalg.norm(f64(y[:3]))


def test_a_step_repeats_to_the_bit():
    theta, x, dy, layer = setup(0.25)
    out = []
    for _ in range(2):
        y, saved = layer.forward(x, 7, 5)
        grad = torch.empty_like(theta)
        out.append((y, layer.backward(dy, saved, grad, 7, 5), grad))
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_training_lowers_the_loss():
    """By more than the batches' own noise: a loss averages over 2 x 512 tokens' squared errors, whose
    relative spread is at most that of one squared normal per token, sqrt(2); four standard deviations
    of the mean are 4 sqrt(2 / 1024) = 0.18."""
    losses = ex.train(d=256, ff=512, tokens=512, steps=25, log=None)
    assert np.isfinite(losses).all() and losses[-1] < (1 - 0.18) * losses[0], losses
    assert dm.device_fault() == 0
