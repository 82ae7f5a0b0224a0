"""What autograd would follow into a call that records nothing is refused, whichever argument it is."""

import pytest
import torch
import torch.autograd.forward_ad as fwAD

import decoupled_momentum_optimizer_gb300 as dm
from decoupled_momentum_optimizer_gb300 import training_ops as ops


def test_row_values_that_require_a_gradient():
    r = torch.ones(4, requires_grad=True)
    with pytest.raises(ValueError, match="rstd requires a gradient"):
        ops._row_values(r, "rstd", 4, r)
    with torch.no_grad():
        assert ops._row_values(r, "rstd", 4, r) == r.data_ptr()
    assert ops._row_values(r.detach(), "rstd", 4, r) == r.data_ptr()


@pytest.mark.gpu
def test_factors_and_weight_gradients_that_require_a_gradient():
    x, w = torch.ones(4, 8, device="cuda"), torch.ones(8, device="cuda")
    rstd = dm.rms_norm(x, w, save=True).rstd
    r, d = rstd.clone().requires_grad_(), w.clone().requires_grad_()
    calls = [(lambda: dm.rms_norm(x, w, rstd=r), "rstd"), (lambda: dm.rms_norm_grad(x, x, w, r), "rstd"),
             (lambda: dm.rms_norm_grad(x, x, w, rstd, dweight=d), "dweight"), (lambda: dm.grad_norm(x, out=r[0]), "out"),
             (lambda: dm.clip_grads(x.clone(), 1.0, norm=r[0]), "norm")]
    for call, name in calls:
        with pytest.raises(ValueError, match=f"{name} requires a gradient"):
            call()
        with torch.no_grad():
            call()


def test_tangents():
    """A dual tensor is refused wherever autograd would follow it, so also under no_grad; not where it does not."""
    x = torch.ones(4)
    ops._unfollowed(x, "x")
    with fwAD.dual_level():
        d = fwAD.make_dual(x, torch.ones(4))
        for t in (d, d[1:]):
            with pytest.raises(ValueError, match="x has a forward-mode tangent"):
                ops._unfollowed(t, "x")
            with torch.no_grad(), pytest.raises(ValueError, match="x has a forward-mode tangent"):
                ops._unfollowed(t, "x")
        ops._unfollowed(x, "x")
        ops._unfollowed(d.detach(), "x")
        ops._unfollowed(fwAD.unpack_dual(d).primal, "x")
        with torch.inference_mode():
            ops._unfollowed(d, "x")
        with pytest.raises(ValueError, match="rstd has a forward-mode tangent"):
            ops._row_values(d, "rstd", 4, d)
    ops._unfollowed(d, "x")


class Doubled(torch.autograd.Function):
    """2 rms_norm(x), with its tangent by the formula."""

    @staticmethod
    def forward(ctx, x, w):
        n = dm.rms_norm(x, w, save=True)
        ctx.save_for_forward(x, w, n.rstd)
        return n.out + n.out

    @staticmethod
    def jvp(ctx, dx, dw):
        x, w, r = ctx.saved_tensors
        xh = x * r[:, None]
        return 2 * w * r[:, None] * (dx - xh * (dx * xh).mean(1, keepdim=True))


@pytest.mark.gpu
def test_calls_with_a_tangent():
    x = torch.randn(4, 8, generator=torch.Generator().manual_seed(1)).cuda()
    w, t = torch.ones(8, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    rstd = dm.rms_norm(x, w, save=True).rstd
    q = dm.fp8_quantize(x)
    calls = [lambda d: dm.rms_norm(d, w), lambda d: dm.rms_norm(x, d[0]), lambda d: dm.rms_norm(x, w, residual=d),
             lambda d: dm.rms_norm_grad(d, x, w, rstd), lambda d: dm.rms_norm_grad(x, x, w, d[:, 0].contiguous()),
             lambda d: dm.embedding(t, d), lambda d: dm.embedding_grad(t, d, 5), lambda d: dm.grad_norm([x, d]),
             lambda d: dm.clip_grads([d], 1.0), lambda d: dm.clip_grads([x], 1.0, out=[d]), lambda d: dm.dropout(d, 0.5, seed=0, step=0),
             lambda d: dm.fp8_quantize(d), lambda d: dm.fp8_linear(d, q)]
    for call in calls:
        call(x.clone())
    with fwAD.dual_level():
        d = fwAD.make_dual(x.clone(), torch.ones(4, 8, device="cuda"))
        for call in calls:
            with pytest.raises(ValueError, match="has a forward-mode tangent"):
                call(d)
            with torch.no_grad(), pytest.raises(ValueError, match="has a forward-mode tangent"):
                call(d)
            call(d.detach().clone())  # some write into it
        r = fwAD.unpack_dual(Doubled.apply(d, w))
    # Against a difference in 64 bits.  f is 2 sqrt(8) times the row's direction, whose Taylor coefficients along h are two
    # Legendre polynomials times (|h| / |v|)^k, here r^k, at most 2 r^k: the difference is off by at most 4 sqrt(8) r (h r)^2
    # and what is smaller by (h r)^2 again.  float32: some twenty roundings of terms up to 2 r (1 + 8).
    h, rmax = 2.0 ** -6, float(rstd.max())
    f = lambda v: 2 * v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt()
    xd = x.double()
    want = (f(xd + h) - f(xd - h)) / (2 * h)
    assert h * rmax < 0.25
    assert bool(((r.tangent.double() - want).abs() <= 12 * h ** 2 * rmax ** 3 + 2.0 ** -15 * rmax).all())
