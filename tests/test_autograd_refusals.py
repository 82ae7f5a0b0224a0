"""What autograd would follow into a call that records nothing is refused, whichever argument it is."""

import pytest
import torch

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
