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


def check_linear_range(x, w, k):
    """fp8_linear of x and w against 64 bits wherever no sum of magnitudes comes near float32's largest
    value; infinite or NaN where the result is above it."""
    m = x.shape[0]
    q = dm.fp8_quantize(w.cuda())
    xv = ref.values(*ref.quantize(x.double().numpy(), "e4m3"), k)
    want, total = ref.product(xv, ref.values(f64(q.codes), f64(q.scales), k))
    got = f64(dm.fp8_linear(x.cuda(), q))
    largest = float(np.finfo(np.float32).max)
    inside = total < largest / 4
    # A block's term and the sum it joins lose half of the smallest step each; the tensor core's sums are
    # not held to float32's subnormal steps.
    tiny = (2 * ((k + 127) // 128) + 4) * 2.0 ** -149 if m <= 40 else 2.0 ** -126
    tol = ref.product_tolerance(total, k) + ref.round_tolerance(want, "f32") + tiny
    assert (np.abs(got - want) <= tol)[inside].all()
    assert not np.isfinite(got[np.abs(want) > 1.01 * largest]).any()
    return inside


@pytest.mark.parametrize("m", [5, 9, 20, 40, 41, 200])
@pytest.mark.parametrize("k", [515, 1700])
def test_linear_between_the_ends_of_the_range(m, k):
    """Tokens and rows of w of every size, and of one size in a block and another in the next: the scales'
    product, or a sum times one of them, leaves float32's range where the result does not."""
    sizes = [2.0 ** e for e in (-124, -70, 0, 70, 123)]
    x, w = normal(m, k, 11), normal(130, k, 12)
    for i, size in enumerate(sizes):
        x[i::5] *= size / x[i::5].abs().max()
        w[i::5] *= size / w[i::5].abs().max()
    x[:, 128:256] *= 2.0 ** -40
    w[:, 128:256] = (w[:, 128:256] * 2.0 ** 40).clamp(-2.0 ** 123, 2.0 ** 123)
    inside = check_linear_range(x, w, k)
    assert 0.5 < inside.mean() < 0.9


@pytest.mark.parametrize("m", [3, 20, 100])
def test_linear_of_small_codes_under_large_scales(m):
    """The scales' product is 2^130 where the result is 2^112, or 0."""
    x, w = torch.zeros(m, 300), torch.zeros(50, 300)
    x[:, 7], x[:, 8] = 448 * 2.0 ** 65, 2.0 ** -9 * 2.0 ** 65
    w[:, 9], w[:25, 8] = 448 * 2.0 ** 65, 2.0 ** -9 * 2.0 ** 65
    got = f64(dm.fp8_linear(x.cuda(), dm.fp8_quantize(w.cuda())))
    assert (got[:, :25] == 2.0 ** 112).all() and (got[:, 25:] == 0).all()


@pytest.mark.parametrize("m", [3, 20, 100])
def test_linear_of_large_values_that_do_not_meet(m):
    """Blocks with float32's largest powers of two in both, opposite zeros: no infinity times zero."""
    x, w = torch.ones(m, 300), torch.zeros(50, 300)
    x[:, 7] = 2.0 ** 127
    w[:, 8], w[:, 200] = 2.0 ** 127, 1.0  # column 8 meets ones whose codes beside 2^127 are 0
    assert (f64(dm.fp8_linear(x.cuda(), dm.fp8_quantize(w.cuda()))) == 1.0).all()


@pytest.mark.parametrize("m,n", [(5, 7), (5, 8), (3000, 1301), (3000, 1304)])
def test_an_empty_sum_leaves_out_as_it_is(m, n):
    """To the bit: -0, subnormal values, NaN with their payloads."""
    out = torch.full((m, n), -0.0, device="cuda")
    out[::2, 3], out[1, 1] = 1e-42, 3.0
    out.view(torch.int32)[2, 2] = 0x7FC12345
    want = out.clone()
    dm.fp8_matmul(dm.Fp8Matrix.empty(m, 0), dm.Fp8Matrix.empty(n, 0), out=out, add=True)
    assert torch.equal(out.view(torch.int32), want.view(torch.int32))


@pytest.mark.parametrize("m,n,k", [(3, 300, 700), (200, 300, 2000), (2100, 1300, 700)])
@pytest.mark.parametrize("pad", [0, 1, 4])
def test_add_keeps_subnormal_values(m, n, k, pad):
    """The addition is float32's with its subnormal values, whichever way the result is written (bulk
    reductions of whole 16-byte units, single elements, the join of parts of k)."""
    x, y = torch.zeros(m, k), torch.zeros(n, k)
    x[:, 5], y[1::2, 5] = 1.0, 2.0 ** -126
    out = torch.empty(m, n + pad, device="cuda")[:, :n]
    out[:, ::2] = torch.tensor([1e-40, -1e-45], device="cuda").repeat(m)[:m, None]
    out[:, 1::2] = -1.5 * 2.0 ** -126  # a subnormal sum
    want = out.clone()
    want[:, 1::2] = -(2.0 ** -127)
    dm.fp8_matmul(dm.fp8_quantize(x.cuda()), dm.fp8_quantize(y.cuda()), out=out, add=True)
    assert torch.equal(out, want)


@pytest.mark.parametrize("item", [0, 13, 16, 23])
def test_linear_ends_when_a_load_of_any_round_never_completes(item):
    """Six row blocks on the first CTA, in two rounds of its groups of warps (16 and 8 loads): every group
    stops as one, in either round, and the next call is right."""
    n, k = 16 * (5 * torch.cuda.get_device_properties(0).multi_processor_count + 3), 2000
    w, x = dm.fp8_quantize(normal(n, k, 21).cuda()), normal(3, k, 22).cuda()
    want = dm.fp8_linear(x, w)
    assert dm.device_fault() == 0
    dm.test_stall_next_launch(item)
    dm.fp8_linear(x, w)
    assert dm.device_fault() == 1
    assert torch.equal(dm.fp8_linear(x, w), want) and dm.device_fault() == 0


@pytest.mark.parametrize("m,n,k,item", [(2100, 1300, 700, 5), (200, 300, 2000, 1), (3, 300, 700, 5)])
def test_matmul_ends_when_one_of_its_last_loads_never_completes(m, n, k, item):
    """The thread that loads has nothing left to ask for by then: it stays until its copies have landed."""
    a, b = dm.fp8_quantize(normal(m, k, 23).cuda()), dm.fp8_quantize(normal(n, k, 24).cuda())
    want = dm.fp8_matmul(a, b)
    assert dm.device_fault() == 0
    dm.test_stall_next_launch(item)
    dm.fp8_matmul(a, b)
    assert dm.device_fault() == 1
    assert torch.equal(dm.fp8_matmul(a, b), want) and dm.device_fault() == 0


def test_tensors_that_require_a_gradient_are_refused():
    """A result without history would end a branch's training without a word."""
    x, r = normal(4, 128, 31).cuda(), normal(4, 128, 32).cuda()
    g = normal(4, 128, 33).cuda().requires_grad_()
    w = dm.fp8_quantize(normal(6, 128, 34).cuda())
    out = torch.empty(4, 6, device="cuda", requires_grad=True)
    calls = [lambda: dm.dropout(g, 0.1, seed=0, step=0), lambda: dm.dropout(x, 0.1, seed=0, step=0, residual=g),
             lambda: dm.dropout(x, 0.1, seed=0, step=0, out=g), lambda: dm.fp8_quantize(g),
             lambda: dm.fp8_quantize(x, gate=g), lambda: dm.fp8_linear(g, w), lambda: dm.fp8_linear(x, w, out=out),
             lambda: dm.fp8_matmul(dm.fp8_quantize(x), w, out=out),
             lambda: dm.dropout(g, 0.1, seed=0, step=0, stream=torch.cuda.current_stream())]
    for call in calls:
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
        with torch.no_grad():
            call()
    assert torch.equal(dm.dropout(g.detach(), 0.1, seed=0, step=0, residual=r),
                       dm.dropout(g.data, 0.1, seed=0, step=0, residual=r))


class Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, seed, step):
        ctx.args = p, seed, step
        return dm.dropout(x, p, seed=seed, step=step, residual=residual)

    @staticmethod
    def backward(ctx, dy):
        p, seed, step = ctx.args
        return dm.dropout(dy, p, seed=seed, step=step), dy, None, None, None


def test_dropout_from_an_autograd_function():
    x, r, w = (normal(9, 130, s).cuda() for s in (35, 36, 37))
    x.requires_grad_(), r.requires_grad_()
    (Dropout.apply(x, r, 0.3, 5, 6) * w).sum().backward()
    keep = torch.from_numpy(ref.keep_mask(9, 130, 0.3, 5, 6, 0)).cuda()
    want = torch.where(keep, w * ref.drop_scale(0.3), torch.zeros_like(w))
    assert torch.allclose(x.grad, want, rtol=2.0 ** -23, atol=0) and torch.equal(r.grad, w)
