"""The order of the embedding gradient's sums: the tokens, their number and the columns decide it, nothing else does."""

import numpy as np
import pytest
import torch

import decoupled_momentum_optimizer_gb300 as dm
from model_ref import draw, guarded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [20, 500, 9000, 70000])
@pytest.mark.parametrize("cols", [40, 768])
def test_the_same_bits_whatever_else_differs(n, cols):
    """Another table length, 32-bit tokens, rows off 16 bytes (other accesses), added to zeros, in rows of tokens."""
    gen = np.random.default_rng(90)
    t = torch.from_numpy((300 * gen.random(n) ** 3).astype(np.int64)).cuda()
    dy = draw(n, cols, "bf16", 91)
    want = dm.embedding_grad(t, dy, 300, scale=1.5)
    assert torch.equal(dm.embedding_grad(t, dy, 70001, scale=1.5)[:300], want)
    assert torch.equal(dm.embedding_grad(t.int(), dy, 300, scale=1.5), want)
    assert torch.equal(dm.embedding_grad(t, dy, out=torch.zeros_like(want), add=True, scale=1.5), want)
    out, fine = guarded(300, cols, "f32", 1, 3)
    odd = torch.empty(n * (cols + 3) + 1, dtype=dy.dtype, device="cuda")[1:].view(n, cols + 3)[:, :cols]
    odd.copy_(dy)
    assert torch.equal(dm.embedding_grad(t, odd, out=out, scale=1.5), want) and fine()
    rows = torch.zeros(n // 10, 17, dtype=torch.int64, device="cuda")
    rows[:, 2:12] = t.view(-1, 10)
    assert torch.equal(dm.embedding_grad(rows[:, 2:12], dy.view(n // 10, 10, cols), 300, scale=1.5), want)
