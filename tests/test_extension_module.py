"""The extension module beside the library: what happens where it is not there, cannot be built or is another torch's."""

import os
import sys
import warnings

import pytest
import torch

import decoupled_momentum_optimizer_gb300 as dm
from decoupled_momentum_optimizer_gb300 import build, training_ops as ops

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


# ---- building it ---------------------------------------------------------------------------------

@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """A module path of the test's own, with an older module there, and the library as it is."""
    build.build()
    path = tmp_path / "_bind_ops.so"
    path.write_bytes(b"")
    os.utime(path, (1, 1))
    monkeypatch.setattr(build, "BIND_PATH", str(path))
    return path


@pytest.mark.parametrize("missing", ["compiler", "CUDA in torch", "torch that loads"])
def test_the_library_is_built_without_the_module(elsewhere, monkeypatch, capfd, missing):
    """What keeps the module from being built is reported; the library is there, an outdated module is not."""
    if missing == "compiler":
        monkeypatch.setenv("CXX", "/nonexistent/c++")
    elif missing == "CUDA in torch":
        monkeypatch.setattr(torch.version, "cuda", None)
    else:
        monkeypatch.setattr(build, "_torch", lambda: True)
        monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == build.LIB_PATH
    assert not elsewhere.exists()
    assert "calls go through ctypes" in capfd.readouterr().err


def test_cuda_headers_beside_an_nvcc_on_the_path(monkeypatch, tmp_path):
    nvcc, header, link = tmp_path / "cuda/bin/nvcc", tmp_path / "cuda/include/cuda_runtime.h", tmp_path / "links/bin/nvcc"
    for p in (nvcc, header, link):
        p.parent.mkdir(parents=True, exist_ok=True)
    nvcc.write_text("#!/bin/sh\n")
    nvcc.chmod(0o755)
    header.write_text("")
    link.symlink_to(nvcc)
    for folder in (nvcc.parent, link.parent):
        monkeypatch.setenv("PATH", str(folder))
        for name in ("nvcc", str(nvcc)):
            include = build._cuda_include(name)
            assert os.path.isabs(include) and os.path.samefile(include, header.parent)
    monkeypatch.setenv("PATH", str(tmp_path))
    assert build._cuda_include("nvcc") is None
