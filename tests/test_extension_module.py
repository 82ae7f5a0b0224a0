"""The extension module beside the library: what happens where it is not there, cannot be built or is another torch's."""

import sys
import warnings

import pytest
import torch

import decoupled_momentum_optimizer_gb300 as dm
from decoupled_momentum_optimizer_gb300 import training_ops as ops

PACKAGE = dm.__name__


@pytest.fixture
def unbound(monkeypatch):
    """The bindings as they are before their first call."""
    ops._extension.cache_clear()
    monkeypatch.setattr(ops, "_bind", ops._Bindings())
    yield monkeypatch
    ops._extension.cache_clear()


def block(monkeypatch):
    """The module cannot be imported."""
    monkeypatch.delattr(dm, "_bind_ops", raising=False)
    monkeypatch.setitem(sys.modules, PACKAGE + "._bind_ops", None)


X, T = torch.ones(4, 8), torch.zeros(4, dtype=torch.int64)
CALLS = [lambda x, t: dm.rms_norm(x, x[0]), lambda x, t: dm.rms_norm_grad(x, x, x[0], x[:, 0].contiguous()),
         lambda x, t: dm.embedding(t, x), lambda x, t: dm.embedding_grad(t, x, 5), lambda x, t: dm.grad_norm([x]),
         lambda x, t: dm.clip_grads([x], 0.5)]


def test_calls_without_the_module_go_on_with_one_warning(unbound):
    """Each call reaches the checks behind the module (here: there is no CPU path); the first one says what is missing."""
    block(unbound)
    with warnings.catch_warnings(record=True) as said:
        warnings.simplefilter("always")
        for call in CALLS + CALLS:
            with pytest.raises(ValueError, match="must be on a CUDA device"):
                call(X, T)
    assert [w.category for w in said] == [RuntimeWarning] and "decoupled_momentum_optimizer_gb300.build" in str(said[0].message)


def tensors(r):
    return [r] if isinstance(r, torch.Tensor) else [t for v in r if v is not None for t in tensors(v)]


@pytest.mark.gpu
def test_results_without_the_module(unbound):
    x, t = torch.randn(4, 8, generator=torch.Generator().manual_seed(1)).cuda(), T.cuda()
    want = [tensors(call(x.clone(), t)) for call in CALLS]
    ops._extension.cache_clear()
    unbound.setattr(ops, "_bind", ops._Bindings())
    block(unbound)
    with pytest.warns(RuntimeWarning, match="ctypes"):
        got = [tensors(call(x.clone(), t)) for call in CALLS]
    assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
