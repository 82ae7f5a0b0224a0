"""What a call writes of the tensors that it is given counts as modified in place: autograd notices a saved one."""

import types

import pytest
import torch

import decoupled_momentum_optimizer_gb300 as dm
from decoupled_momentum_optimizer_gb300 import training_ops as ops


def test_counts():
    a, b = torch.ones(2), torch.ones(2)
    with torch.inference_mode():
        c = torch.ones(2)
    ops._written(a, None, b, c)
    assert a._version == 1 and b._version == 1
    q = types.SimpleNamespace(codes=a, scales=b)  # whatever has a quantized matrix's buffers
    ops._written(q, q)
    assert a._version == 3 and b._version == 3


class Declines:
    def __getattr__(self, name):
        return lambda *args: NotImplemented


def calls():
    """(name, a call without results of its own, the given tensors that it writes, those that it reads)."""
    x, w, t = torch.randn(4, 8, device="cuda"), torch.ones(8, device="cuda"), torch.tensor([1, 2, 1, 9], device="cuda")
    new = lambda *s: torch.ones(*(s or (4, 8)), device="cuda")
    r, o, s, d, k, g, n = new(), new(), new(4), new(8), new(4, 4), new(10, 8), new(1)
    q, p = dm.Fp8Matrix.empty(4, 8), dm.Fp8Matrix.empty(8, 4)
    xq = dm.fp8_quantize(x)
    gs, to = [new(), new(3)], [new(), new(3)]
    yield "norm", lambda: dm.rms_norm(x, w, residual=r, out=o, total=r, rstd=s), [o, r, s], [x, w]
    yield "norm into codes", lambda: dm.rms_norm(x, w, form="both", quantized=(q, p)), [q.codes, q.scales, p.codes, p.scales], [x]
    yield "norm without results given", lambda: dm.rms_norm(x, w, residual=r, save=True), [], [x, w, r]
    yield "norm gradient", lambda: dm.rms_norm_grad(x, r, w, s, past=x, out=o, dweight=d, add=True), [o, d], [x, r, w, s]
    yield "embedding", lambda: dm.embedding(t, g, out=o), [o], [t, g]
    yield "embedding gradient", lambda: dm.embedding_grad(t, x, out=g, add=True), [g], [t, x]
    yield "grad norm", lambda: dm.grad_norm(gs, out=n), [n], gs
    yield "clipping", lambda: dm.clip_grads(gs, 1.0), gs, []
    yield "clipping of one", lambda: dm.clip_grads(o, 1.0), [o], []
    yield "clipping into others", lambda: dm.clip_grads(gs, 1.0, out=to), to, gs
    yield "clipping by a norm", lambda: dm.clip_grads(gs, 1.0, norm=n), gs, [n]
    yield "dropout", lambda: dm.dropout(x, 0.5, seed=0, step=0, out=o), [o], [x]
    yield "quantize", lambda: dm.fp8_quantize(x, out=q), [q.codes, q.scales], [x]
    yield "product", lambda: dm.fp8_matmul(xq, xq, out=k, add=True), [k], [xq.codes]
    yield "linear", lambda: dm.fp8_linear(x, xq, out=k), [k], [x, xq.codes]


@pytest.mark.gpu
@pytest.mark.parametrize("way", ["extension", "ctypes", "stream"])
def test_calls_count_what_they_write(way, monkeypatch):
    dm.init(0)
    if way == "ctypes":
        monkeypatch.setattr(ops, "_bind", Declines())
    for name, call, written, read in calls():
        torch.cuda.synchronize()
        before = [t._version for t in written + read]
        if way == "stream":
            with torch.cuda.stream(torch.cuda.Stream()):
                call()
        else:
            call()
        torch.cuda.synchronize()
        after = [t._version for t in written + read]
        assert [a - b for a, b in zip(after, before)] == [1] * len(written) + [0] * len(read), name
    x = torch.randn(4, 8, device="cuda")
    with pytest.raises(dm.DemoError):  # nothing is written
        dm.rms_norm(x, x[0], eps=-1.0, out=x)
    assert x._version == 0
    with torch.inference_mode():
        y = torch.ones(4, device="cuda")
        dm.clip_grads(y, 0.5)
    dm.clip_grads(y, 0.25)
    assert float(y.norm()) < 0.2500001


@pytest.mark.gpu
def test_autograd_notices_a_saved_tensor_that_was_overwritten():
    leaf = torch.ones(4, 8, device="cuda", requires_grad=True)
    h = leaf * 2
    y = (h * h).sum()  # saves h
    with torch.no_grad():
        dm.clip_grads(h, 0.5)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    h = leaf * 2
    y = (h * h).sum()
    with torch.no_grad():
        dm.clip_grads(h, 0.5, out=torch.empty_like(h))
    y.backward()
    assert bool((leaf.grad == 8).all())
