"""The training operators where their results are easily wrong: scales that are no power of two, values
next to the ends of float32's range, sums over nothing, waits that run out."""

import numpy as np
import pytest
import torch

import decoupled_momentum_optimizer_gb300 as dm
import train_ref as ref

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def normal(rows, k, seed):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(rows, k, generator=gen) * torch.exp(torch.randn(rows, k, generator=gen))


# One CTA per tile, k cut into parts, pairs of CTAs.
PRODUCTS = [(3, 300, 700), (40, 130, 515), (200, 300, 2000), (2100, 1300, 700)]
NO_SCALES = [3.0, 1.0 + 2.0 ** -23, 2.0 ** 127 * 1.5, -1.0, -0.0, 2.0 ** -127, float("inf"), float("nan")]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
@pytest.mark.parametrize("scale", NO_SCALES)
def test_matmul_with_a_scale_that_is_no_power_of_two(m, n, k, scale):
    """Its row or column of the result is NaN, the others are what they were."""
    a, b = dm.fp8_quantize(normal(m, k, 1).cuda()), dm.fp8_quantize(normal(n, k, 2).cuda())
    want = dm.fp8_matmul(a, b, dtype=torch.float32)
    a.scales[1, 2] = scale
    b.scales[0, 5], b.scales[-1, n - 1] = scale, scale
    got = dm.fp8_matmul(a, b, dtype=torch.float32)
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    bad[2], bad[:, 5], bad[:, n - 1] = True, True, True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("m", [1, 9, 20, 40, 41, 200])
@pytest.mark.parametrize("scale", NO_SCALES)
def test_linear_with_a_scale_that_is_no_power_of_two(m, scale):
    """The same for every number of rows: NaN in the columns that the scale belongs to."""
    w, x = dm.fp8_quantize(normal(150, 700, 3).cuda()), normal(m, 700, 4).cuda()
    want = dm.fp8_linear(x, w)
    w.scales[0, 5], w.scales[3, 14], w.scales[-1, 149] = scale, scale, scale
    got = dm.fp8_linear(x, w)
    bad = torch.zeros(m, 150, dtype=torch.bool, device="cuda")
    bad[:, [5, 14, 149]] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("m", [3, 100])
def test_scales_of_zero_blocks_and_past_the_rows(m):
    """A scale of 0 on codes of 0 adds nothing, and what follows the last row up to the scales' stride is not used."""
    x, w = normal(m, 300, 5), normal(130, 300, 6)
    x[1, 128:256], w[7, :128] = 0.0, 0.0
    a, b = dm.fp8_quantize(x.cuda()), dm.fp8_quantize(w.cuda())
    want, few = dm.fp8_matmul(a, b), dm.fp8_linear(x.cuda(), b)
    a.scales[1, 1], b.scales[0, 7] = 0.0, 0.0
    a.scales[:, m:], b.scales[:, 130:] = 3.0, float("nan")
    assert torch.equal(dm.fp8_matmul(a, b), want) and torch.equal(dm.fp8_linear(x.cuda(), b), few)


def test_check_of_given_scales():
    q = dm.fp8_quantize(normal(6, 300, 7).cuda())
    q.scales[1, 3], q.scales[:, 6:] = 0.0, 3.0  # allowed; past the rows
    dm.Fp8Matrix(q.codes, q.scales, 300, check=True)
    for scale in NO_SCALES:
        s = q.scales.clone()
        s[2, 4] = scale
        dm.Fp8Matrix(q.codes, s, 300)
        with pytest.raises(ValueError, match="powers of two"):
            dm.Fp8Matrix(q.codes, s, 300, check=True)
