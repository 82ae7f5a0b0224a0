"""The extension module's calls beside the ctypes ones: the same results, the same refusals, and no call that one
of them takes and the other does not."""

import pytest
import torch

import decoupled_momentum_optimizer_gb300 as dm
from decoupled_momentum_optimizer_gb300 import training_ops as ops
from model_ref import DT, draw

pytestmark = pytest.mark.gpu


class Declines:
    """In the extension module's place: takes no call."""

    def __getattr__(self, name):
        return lambda *args: NotImplemented


class Counts:
    """The extension module, counting the calls that it takes."""

    def __init__(self, inner):
        self.inner, self.taken, self.left = inner, 0, 0

    def __getattr__(self, name):
        def call(*args):
            r = getattr(self.inner, name)(*args)
            if r is NotImplemented:
                self.left += 1
            else:
                self.taken += 1
            return r
        return call


@pytest.fixture
def through(monkeypatch):
    """through("ctypes" or "extension", f): f's result on that way, which has to have been taken."""
    bind = ops._bind
    dm.init(0)  # a call before that goes through ctypes, which initialises the library

    def run(way, f):
        counts = Counts(bind)
        with monkeypatch.context() as m:
            m.setattr(ops, "_bind", Declines() if way == "ctypes" else counts)
            r = f()
        assert way == "ctypes" or (counts.taken > 0 and counts.left == 0)
        return r
    return run


def flat(r):
    """The tensors of a result."""
    if isinstance(r, torch.Tensor):
        return [r]
    if isinstance(r, dm.Fp8Matrix):
        return [r.codes.view(torch.uint8), r.scales, torch.tensor(r.shape), torch.tensor(r.tiles)]
    return [] if r is None else [t for v in r for t in flat(v)]


def same(through, f):
    a, b = through("extension", f), through("ctypes", f)
    x, y = flat(a), flat(b)
    assert len(x) == len(y) and type(a) is type(b)
    for p, q in zip(x, y):
        assert p.shape == q.shape and p.dtype == q.dtype and torch.equal(p, q)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("form", [None, "rows", "cols", "both"])
@pytest.mark.parametrize("residual,values,save", [(False, True, False), (True, False, True), (True, True, True)])
def test_norm(through, dtype, pad, form, residual, values, save):
    x, r, w = draw(9, 200, dtype, 1, pad=pad), draw(9, 200, dtype, 2), draw(1, 200, "f32", 3)[0]
    if not (values or form or save):
        pytest.skip("nothing is asked for")
    same(through, lambda: dm.rms_norm(x, w, residual=r if residual else None, values=values, form=form, save=save, fmt="e5m2"))


def test_norm_into_given_buffers(through):
    x, r, w = draw(9, 200, "bf16", 1), draw(9, 200, "bf16", 2), draw(1, 200, "bf16", 3)[0]

    def f():
        o, t, s = torch.empty_like(x), torch.empty(9, 207, dtype=x.dtype, device="cuda")[:, :200], torch.empty(9, device="cuda")
        n = dm.rms_norm(x, w, residual=r, out=o, total=t, rstd=s, eps=1)
        assert n.out is o and n.total is t and n.rstd is s and n.quantized is None
        return n
    same(through, f)
    same(through, lambda: dm.rms_norm(x.view(3, 3, 200), w, residual=r.view(3, 3, 200)))
    same(through, lambda: dm.rms_norm(x[0], w, save=True))
    n = through("extension", lambda: dm.rms_norm(x, w))
    assert n.total is x and n.rstd is None


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("past,add,weight_grad", [(False, False, True), (True, True, True), (True, False, False)])
def test_norm_grad(through, dtype, past, add, weight_grad):
    s, dy, w = draw(70, 200, dtype, 4), draw(70, 200, dtype, 5, pad=5), draw(1, 200, "f32", 6)[0]
    r = dm.rms_norm(s, w, save=True).rstd
    same(through, lambda: dm.rms_norm_grad(dy, s, w, r, past=s if past else None, add=add, weight_grad=weight_grad,
                                           dweight=torch.ones(200, device="cuda") if add else None))
    out, dw = torch.empty_like(s), torch.empty(200, device="cuda")
    got = through("extension", lambda: dm.rms_norm_grad(dy, s, w, r, out=out, dweight=dw))
    assert got[0] is out and got[1] is dw


@pytest.mark.parametrize("idx", [torch.int32, torch.int64])
def test_embedding(through, idx):
    t, table = torch.tensor([[1, 5, -1], [0, 9, 99]], dtype=idx, device="cuda"), draw(10, 40, "f32", 7, pad=2)
    dy = draw(6, 40, "bf16", 8).view(2, 3, 40)
    same(through, lambda: dm.embedding(t, table, scale=2, dtype=torch.bfloat16))
    same(through, lambda: dm.embedding(t, table))
    same(through, lambda: dm.embedding(t, table, out=torch.empty(2, 3, 40, dtype=torch.float16, device="cuda")))
    same(through, lambda: dm.embedding_grad(t, dy, 10, scale=0.5))
    same(through, lambda: dm.embedding_grad(t, dy, out=torch.ones(10, 43, device="cuda")[:, :40], add=True))
    same(through, lambda: dm.embedding(t[0, 1], table))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_clipping(through, dtype):
    g = [draw(5, 300, dtype, 9), draw(1, 7, dtype, 10)[0], torch.empty(0, dtype=DT[dtype], device="cuda")]
    same(through, lambda: dm.grad_norm(g))
    same(through, lambda: dm.grad_norm(g[0], out=torch.empty(1, device="cuda")))

    def into(odt, **kw):
        out = tuple(torch.zeros(v.shape, dtype=odt, device="cuda") for v in g)
        return [dm.clip_grads(g, 0.5, out=out, **kw), out]

    def in_place(**kw):
        c = [v.clone() for v in g]
        return [dm.clip_grads(c, 0.5, **kw), c]

    for f in (lambda: into(DT[dtype]), lambda: into(torch.float32), in_place,
              lambda: in_place(norm=torch.tensor(3.0, device="cuda"))):
        same(through, f)


def test_refused_alike(through):
    x, w, t = draw(8, 64, "f32", 11), draw(1, 64, "f32", 12)[0], torch.zeros(8, dtype=torch.int64, device="cuda")
    g, r = x.clone().requires_grad_(), torch.ones(8, device="cuda")
    calls = [lambda: dm.rms_norm(g, w), lambda: dm.rms_norm(x, w, eps=-1.0), lambda: dm.rms_norm(x, w[:5]), lambda: dm.rms_norm(x, 3),
             lambda: dm.rms_norm(x, w, form="diagonal"), lambda: dm.rms_norm(x, w, fmt="e3m4"), lambda: dm.rms_norm(x, w, values=False),
             lambda: dm.rms_norm(x.cpu(), w), lambda: dm.rms_norm(x, w.cpu()), lambda: dm.rms_norm(x, w, residual=x[:4]),
             lambda: dm.rms_norm(x, w, out=x[:, :63]), lambda: dm.rms_norm(x, w, out=x.t()),
             lambda: dm.rms_norm_grad(x, x, w, r, add=True), lambda: dm.rms_norm_grad(x, x, w, r.double()),
             lambda: dm.rms_norm_grad(x, x, w, r, dweight=w), lambda: dm.embedding(t, x[0]), lambda: dm.embedding(t.float(), x),
             lambda: dm.embedding(t, x, scale=1e300), lambda: dm.embedding(t, x, dtype=torch.int8), lambda: dm.embedding(t, x, out=x),
             lambda: dm.embedding_grad(t, x), lambda: dm.embedding_grad(t, x, -3), lambda: dm.embedding_grad(t[:5], x, 4),
             lambda: dm.grad_norm([]), lambda: dm.grad_norm([x, x.half()]), lambda: dm.grad_norm(3), lambda: dm.clip_grads(x, -1.0),
             lambda: dm.clip_grads([x, x], 1.0), lambda: dm.clip_grads(x, 1.0, out=w), lambda: dm.clip_grads([x, g], 1.0)]
    for f in calls:
        raised = []
        for call in (lambda: through("ctypes", f), f):
            with pytest.raises((ValueError, TypeError, AttributeError, RuntimeError)) as e:
                call()
            raised.append((e.type, str(e.value)))
        assert raised[0] == raised[1]


def test_another_current_device_or_stream():
    x, w = draw(8, 64, "f32", 13), draw(1, 64, "f32", 14)[0]
    want = dm.rms_norm(x, w).out
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = dm.rms_norm(x, w).out
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    with torch.inference_mode():
        assert torch.equal(dm.rms_norm(x, w).out, want)
