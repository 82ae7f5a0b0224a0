"""The embedding gradient of more positions than are sorted at one time, into tables longer than what is filled meanwhile.

The first run's sums write 0 to the rows behind the filled ones that its own tokens do not name; the later runs add.
"""

import numpy as np
import pytest
import torch

import decoupled_momentum_optimizer_gb300 as dm
from model_ref import draw, f64

pytestmark = pytest.mark.gpu

RUN = 65536


@pytest.mark.parametrize("cols,pad", [(256, 0), (301, 0), (256, 4)])
def test_rows_that_only_a_later_run_names(cols, pad):
    """Rows past the filled ones: named by the first run alone, the second alone, both, neither; over NaN."""
    n, vocab = 70001, (200 << 20) // (4 * cols) + 3  # 200 MB, of 146 that are filled
    gen = np.random.default_rng(92)
    t = gen.integers(0, vocab, n)
    end = np.arange(vocab - 4000, vocab)
    first, second, both = end[0::4], end[1::4], end[2::4]
    t[(t >= vocab - 4000)] -= 4000
    t[:1000], t[1000:2000] = first, both
    t[RUN:RUN + 1000], t[RUN + 1000:RUN + 2000], t[RUN + 2000:RUN + 2500] = second, both, second[:500]
    dy = draw(n, cols, "bf16", 93)
    buf = torch.full((vocab, cols + pad), float("nan"), device="cuda")
    buf[:, cols:] = 5.0
    got = dm.embedding_grad(torch.from_numpy(t).cuda(), dy, out=buf[:, :cols])
    names, inverse, count = np.unique(t, return_inverse=True, return_counts=True)
    d = f64(dy)
    order = np.argsort(inverse, kind="stable")
    starts = np.concatenate([[0], np.cumsum(count)[:-1]])
    want, mag = np.add.reduceat(d[order], starts), np.add.reduceat(np.abs(d[order]), starts)
    # an addition a row, one more for the second run, the product with the scale
    tol = (count[:, None] + 3) * 2.0 ** -24 * mag
    assert (np.abs(f64(got[torch.from_numpy(names).cuda()]) - want) <= tol).all()
    absent = torch.ones(vocab, dtype=torch.bool, device="cuda")
    absent[torch.from_numpy(names).cuda()] = False
    assert bool(absent[-4000:][3::4].all()) and not bool(got[absent].any())
    assert not bool(torch.isnan(got).any()) and bool((buf[:, cols:] == 5.0).all())
