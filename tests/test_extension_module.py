"""The extension module beside the library: what happens where it is not there, cannot be built or is another torch's."""

import os
import sys
import sysconfig
import types
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


def test_a_module_for_another_torch_is_left_alone(unbound):
    """It can be imported, and would read tensors by another layout: it takes no call."""
    def call(*args):
        raise AssertionError("the module was called")

    stale = types.ModuleType(PACKAGE + "._bind_ops")
    stale.rms_norm, stale.torch = call, "1.0 abc"
    unbound.setattr(dm, "_bind_ops", stale, raising=False)
    unbound.setitem(sys.modules, stale.__name__, stale)
    for torch_of in ("1.0 abc", None):
        if torch_of is None:
            del stale.torch
        ops._extension.cache_clear()
        unbound.setattr(ops, "_bind", ops._Bindings())
        with pytest.warns(RuntimeWarning, match="no extension module for this torch"):
            with pytest.raises(ValueError, match="must be on a CUDA device"):
                dm.rms_norm(X, X[0])


def test_the_module_names_its_torch(unbound):
    build.build()
    if not os.path.exists(build.BIND_PATH):
        pytest.skip("the module could not be built here")
    assert ops._extension().torch == build.torch_tag(torch)


# ---- building it ---------------------------------------------------------------------------------

@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """A module path of the test's own, with an older module there, and the library as it is."""
    build.build()
    path = tmp_path / "_bind_ops.so"
    path.write_bytes(b"")
    os.utime(path, (1, 1))
    monkeypatch.setattr(build, "BIND_PATH", str(path))
    monkeypatch.setattr(build, "BIND_STAMP", str(tmp_path / "torch.txt"))
    return path


def test_the_module_is_built_anew_for_another_torch(elsewhere, monkeypatch, tmp_path):
    """The one and only reason here: its own torch is another than the one installed."""
    built = []

    def bind(verbose):
        built.append(1)
        (tmp_path / "torch.txt").write_text(build._torch())

    monkeypatch.setattr(build, "_bind", bind)
    os.utime(elsewhere)
    (tmp_path / "torch.txt").write_text("__version__ = '1.0'")
    build.build(), build.build()
    assert len(built) == 1
    (tmp_path / "torch.txt").unlink()  # not known: anew
    build.build(), build.build()
    assert len(built) == 2 and build._torch() != "__version__ = '1.0'"


def test_a_module_is_of_one_interpreter():
    assert build.BIND_PATH.endswith(sysconfig.get_config_var("EXT_SUFFIX"))


@pytest.mark.parametrize("missing", ["compiler", "CUDA in torch", "torch that loads"])
def test_the_library_is_built_without_the_module(elsewhere, monkeypatch, capfd, missing):
    """What keeps the module from being built is reported; the library is there, an outdated module is not."""
    if missing == "compiler":
        monkeypatch.setenv("CXX", "/nonexistent/c++")
    elif missing == "CUDA in torch":
        monkeypatch.setattr(torch.version, "cuda", None)
    else:
        monkeypatch.setattr(build, "_torch", lambda: "2")
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
