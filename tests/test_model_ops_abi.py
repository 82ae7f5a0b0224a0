"""Refusals and sizes of the norm, embedding and clipping calls without a GPU: every check runs before any
CUDA call, and valid arguments stop at the device check on a machine without one."""

import ctypes

import pytest
import torch

import model_ref as mr

OK, EINVAL, EALIGN, ENODEV, ENOTINIT, ENOSPACE = 0, -1, -2, -3, -5, -6
NODEV = (ENOTINIT, ENODEV)


@pytest.fixture(scope="module")
def L():
    from decoupled_momentum_optimizer_gb300 import build

    build.build()
    import decoupled_momentum_optimizer_gb300 as dm

    if torch.cuda.is_available():
        pytest.skip("made-up pointers: only where no kernel can be reached")
    return dm.lib()


def p(a):
    return ctypes.c_void_p(a)


def norm(L, **kw):
    a = dict(x=p(0x100000), ldx=300, res=None, ldr=300, dtype=1, w=p(0x80000), wd=0, rows=200, cols=300, eps=1e-6, tot=None,
             ldt=300, out=p(0x200000), ldo=300, rstd=None, fmt=0, cr=None, sr=None, cc=None, sc=None)
    a.update(kw)
    return L.demo_rms_norm(a["x"], a["ldx"], a["res"], a["ldr"], a["dtype"], a["w"], a["wd"], a["rows"], a["cols"], a["eps"],
                           a["tot"], a["ldt"], a["out"], a["ldo"], a["rstd"], a["fmt"], a["cr"], a["sr"], a["cc"], a["sc"], None)


def test_norm_refusals(L):
    every = dict(res=p(0x300000), tot=p(0x400000), rstd=p(0x500000), cr=p(0x600000), sr=p(0x700000), cc=p(0x800000),
                 sc=p(0x900000))
    assert norm(L) in NODEV and norm(L, **every) in NODEV
    for bad in (dict(dtype=3), dict(wd=2), dict(wd=-1), dict(dtype=0, wd=1), dict(rows=-1), dict(cols=-1), dict(cols=32769),
                dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(w=None),
                dict(fmt=2), dict(out=None), dict(ldo=299), dict(ldx=-1), dict(tot=p(0x400000)), dict(cr=p(0x600000)),
                dict(sc=p(0x600000)), dict(rows=1 << 31), dict(rows=1 << 30, ldx=0), dict(out=p(0x100002)),
                dict(out=p(0x80000)), dict(rstd=p(0x200000)), dict(rstd=p(0x100000))):
        assert norm(L, **bad) == EINVAL, bad
    for bad in (dict(rstd=None), dict(tot=None), dict(ldt=299), dict(tot=p(0x200000)), dict(out=p(0x100000)),
                dict(out=p(0x300000)), dict(rstd=p(0x400000)), dict(cr=p(0x100000)), dict(sr=p(0x300000)),
                dict(cc=p(0x600010)), dict(sc=p(0x80000)), dict(cc=p(0x400000))):
        assert norm(L, **{**every, **bad}) == EINVAL, bad
    for bad in (dict(x=p(0x100001)), dict(w=p(0x80002)), dict(out=p(0x200001)), dict(rstd=p(0x500002))):
        assert norm(L, **bad) == EALIGN, bad
    for bad in (dict(cr=p(0x600008)), dict(sc=p(0x900004)), dict(tot=p(0x400001)), dict(res=p(0x300001))):
        assert norm(L, **{**every, **bad}) == EALIGN, bad
    # the sum in an input's place; the result too, unless the column form reads the sum again
    assert norm(L, **{**every, "tot": p(0x300000)}) in NODEV and norm(L, **{**every, "tot": p(0x100000)}) in NODEV
    assert norm(L, out=p(0x100000)) in NODEV and norm(L, out=p(0x100000), ldo=301) == EINVAL
    assert norm(L, res=p(0x300000), out=p(0x300000)) in NODEV
    assert norm(L, rows=0) == OK and norm(L, cols=0, x=None) == OK
    assert norm(L, out=None, rstd=p(0x500000)) in NODEV and norm(L, ldx=0) in NODEV


def grad(L, **kw):
    a = dict(dy=p(0x100000), ldd=300, tot=p(0x200000), ldt=300, dtype=1, w=p(0x80000), wd=0, rstd=p(0x90000), rows=200, cols=300,
             past=p(0x300000), ldp=300, dx=p(0x400000), ldx=300, dw=p(0x500000), add=0, work=p(0x600000), bytes=None)
    a.update(kw)
    if a["bytes"] is None:
        a["bytes"] = L.demo_rms_norm_grad_workspace(a["rows"], a["cols"])
    return L.demo_rms_norm_grad(a["dy"], a["ldd"], a["tot"], a["ldt"], a["dtype"], a["w"], a["wd"], a["rstd"], a["rows"], a["cols"],
                                a["past"], a["ldp"], a["dx"], a["ldx"], a["dw"], a["add"], a["work"], a["bytes"], None)


def test_norm_grad_refusals(L):
    assert grad(L) in NODEV and grad(L, add=1) in NODEV and grad(L, past=None) in NODEV
    for bad in (dict(dtype=-1), dict(wd=2), dict(rows=-1), dict(cols=32769), dict(add=2), dict(dy=None), dict(tot=None),
                dict(w=None), dict(rstd=None), dict(dx=None), dict(ldx=299), dict(ldd=-1), dict(work=None),
                dict(dx=p(0x100002)), dict(dx=p(0x80000)), dict(dx=p(0x90000)), dict(dw=p(0x400000)), dict(dw=p(0x80000)),
                dict(work=p(0x400000)), dict(work=p(0x500000)), dict(work=p(0x300000)), dict(dw=p(0x300000))):
        assert grad(L, **bad) == EINVAL, bad
    assert grad(L, bytes=200 * 300 * 4 - 1) == ENOSPACE
    for bad in (dict(dy=p(0x100001)), dict(rstd=p(0x90002)), dict(dw=p(0x500002)), dict(work=p(0x600004)), dict(past=p(0x300001))):
        assert grad(L, **bad) == EALIGN, bad
    for place in (0x100000, 0x200000, 0x300000):
        assert grad(L, dx=p(place)) in NODEV
    assert grad(L, dw=None, work=None, bytes=0) in NODEV and grad(L, rows=1, work=None) in NODEV
    assert grad(L, cols=0) == OK and grad(L, rows=0, add=1) == OK and grad(L, rows=0, dw=None) == OK
    assert grad(L, rows=0) in NODEV  # writes zeros
    ws = L.demo_rms_norm_grad_workspace
    assert ws(200, 300) == 240000 and ws(100000, 300) == 256 * 1200
    assert ws(1, 300) == ws(0, 300) == ws(-5, 3) == ws(5, 0) == ws(5, 32769) == 0


def test_bindings_refuse_cpu_tensors():
    import decoupled_momentum_optimizer_gb300 as dm

    x, w, r = torch.zeros(4, 8), torch.ones(8), torch.ones(4)
    for call in (lambda: dm.rms_norm(x, w), lambda: dm.rms_norm_grad(x, x, w, r)):
        with pytest.raises(ValueError, match="no CPU path"):
            call()


def test_reference_norm_is_the_formula():
    """The reference's float32 products against the 64-bit result: three roundings."""
    s, w = mr.f64(mr.draw(7, 33, "f32", 1, device="cpu")), mr.f64(mr.draw(1, 33, "f32", 2, device="cpu"))[0]
    r = mr.norm_rstd(s, 1e-6)
    want = s * r[:, None] * w
    assert (abs(mr.norm_values(s, r.astype("f4"), w) - want) <= 3.01 * 2.0 ** -24 * abs(want)).all()


def lookup(L, **kw):
    a = dict(t=p(0x10000), tb=8, tr=1, tc=100, ldt=100, tab=p(0x100000), ld=300, td=0, vocab=50, cols=300, scale=1.0,
             out=p(0x200000), ldo=300, od=1)
    a.update(kw)
    return L.demo_embedding(a["t"], a["tb"], a["tr"], a["tc"], a["ldt"], a["tab"], a["ld"], a["td"], a["vocab"], a["cols"],
                            a["scale"], a["out"], a["ldo"], a["od"], None)


def test_embedding_refusals(L):
    assert lookup(L) in NODEV and lookup(L, tb=4, t=p(0x10004)) in NODEV and lookup(L, tr=5, tc=20, ldt=0) in NODEV
    for bad in (dict(tb=2), dict(tr=-1), dict(tc=-1), dict(t=None), dict(ldt=-1), dict(td=3), dict(od=-1), dict(vocab=-1),
                dict(cols=-1), dict(vocab=1 << 31), dict(scale=float("nan")), dict(scale=float("inf")), dict(tab=None),
                dict(out=None), dict(ldo=299), dict(ld=-1), dict(out=p(0x100010)), dict(out=p(0x10000)),
                dict(tr=1 << 20, tc=1 << 20), dict(cols=1 << 30, tc=1 << 20), dict(tr=1 << 20, tc=4, ldt=1 << 30)):
        assert lookup(L, **{"tr": 2, **bad} if "ldt" in bad else bad) == EINVAL, bad
    for bad in (dict(t=p(0x10004)), dict(tab=p(0x100002)), dict(out=p(0x200001))):
        assert lookup(L, **bad) == EALIGN, bad
    assert lookup(L, tc=0, t=None) == OK and lookup(L, cols=0) == OK and lookup(L, vocab=0, tab=None) in NODEV


def embed_grad(L, **kw):
    a = dict(t=p(0x10000), tb=8, tr=1, tc=1000, ldt=1000, dy=p(0x100000), ldd=300, dt=1, vocab=50, cols=300, scale=1.0,
             g=p(0x800000), ldg=300, add=0, work=p(0x900000), bytes=None)
    a.update(kw)
    if a["bytes"] is None:
        a["bytes"] = L.demo_embedding_grad_workspace(max(a["tr"], 0) * max(a["tc"], 0), a["cols"])
    return L.demo_embedding_grad(a["t"], a["tb"], a["tr"], a["tc"], a["ldt"], a["dy"], a["ldd"], a["dt"], a["vocab"], a["cols"],
                                 a["scale"], a["g"], a["ldg"], a["add"], a["work"], a["bytes"], None)


def test_embedding_grad_refusals(L):
    assert embed_grad(L) in NODEV and embed_grad(L, add=1) in NODEV
    for bad in (dict(tb=1), dict(tr=-1), dict(t=None), dict(dt=3), dict(vocab=-1), dict(cols=-1), dict(add=2),
                dict(scale=float("nan")), dict(dy=None), dict(g=None), dict(ldg=299), dict(work=None), dict(g=p(0x100000)),
                dict(g=p(0x10000)), dict(work=p(0x800000)), dict(work=p(0x100000)), dict(work=p(0x10000)),
                dict(vocab=1 << 30, cols=1 << 20)):
        assert embed_grad(L, **bad) == EINVAL, bad
    need = L.demo_embedding_grad_workspace(1000, 300)
    assert embed_grad(L, bytes=need - 1) == ENOSPACE
    for bad in (dict(t=p(0x10004)), dict(dy=p(0x100001)), dict(g=p(0x800002)), dict(work=p(0x900008))):
        assert embed_grad(L, **bad) == EALIGN, bad
    assert embed_grad(L, vocab=0, g=None) == OK and embed_grad(L, cols=0) == OK
    assert embed_grad(L, tc=0, add=1) == OK and embed_grad(L, tc=0, dy=None, work=None) in NODEV
    ws = L.demo_embedding_grad_workspace
    # keys, positions, two parts of 512 columns for each of 125 pieces of 8
    assert need == 4000 + 2000 + 125 * 2 * 512 * 4
    assert ws(33, 300) == 144 + 80 + 5 * 2 * 512 * 4 and ws(32, 300) == ws(1, 300) == 0
    assert embed_grad(L, tc=32, work=None) in NODEV and ws(0, 5) == ws(-1, 5) == ws(5, 0) == 0
    assert ws(1 << 30, 2048) == ws(65536, 2048) == 65536 * 6 + 2048 * 2 * 2048 * 4


def test_bindings_of_tokens_refuse_cpu_tensors():
    import decoupled_momentum_optimizer_gb300 as dm

    t, x = torch.zeros(4, dtype=torch.int64), torch.zeros(4, 8)
    for call in (lambda: dm.embedding(t, x), lambda: dm.embedding_grad(t, x, 4)):
        with pytest.raises(ValueError, match="no CPU path"):
            call()


def arrays(ptrs, sizes):
    return (ctypes.c_void_p * len(ptrs))(*ptrs), (ctypes.c_int64 * len(sizes))(*sizes)


def clip(L, ptrs=(0x100000, 0x200000), sizes=(1000, 2000), out=None, **kw):
    a = dict(count=len(ptrs), dt=0, od=None, mx=1.0, norm=p(0x50000), given=0, work=p(0x60000), bytes=None)
    a.update(kw)
    g, n = arrays(ptrs, sizes)
    o = arrays(out, sizes)[0] if out is not None else None
    if a["bytes"] is None:
        a["bytes"] = L.demo_grad_workspace(max(a["count"], 0))
    if a["od"] is None:
        a["od"] = a["dt"]
    return L.demo_clip_grads(a["count"], g, n, a["dt"], o, a["od"], a["mx"], a["norm"], a["given"], a["work"], a["bytes"], None)


def grad_norm(L, ptrs=(0x100000, 0x200000), sizes=(1000, 2000), **kw):
    a = dict(count=len(ptrs), dt=0, norm=p(0x50000), work=p(0x60000), bytes=1 << 20)
    a.update(kw)
    g, n = arrays(ptrs, sizes)
    return L.demo_grad_norm(a["count"], g, n, a["dt"], a["norm"], a["work"], a["bytes"], None)


def test_clip_refusals(L):
    assert clip(L) in NODEV and grad_norm(L) in NODEV
    for bad in (dict(count=-1), dict(dt=3), dict(norm=None), dict(work=None), dict(norm=p(0x100010)), dict(norm=p(0x60010)),
                dict(work=p(0x200000))):
        assert clip(L, **bad) == EINVAL and grad_norm(L, **bad) == EINVAL, bad
    for bad in (dict(mx=-1.0), dict(mx=float("nan")), dict(given=2), dict(od=1), dict(dt=1, od=2), dict(od=0, dt=1)):
        assert clip(L, **bad) == EINVAL, bad
    for bad in (dict(norm=p(0x50002)), dict(work=p(0x60008))):
        assert clip(L, **bad) == EALIGN and grad_norm(L, **bad) == EALIGN, bad
    assert clip(L, ptrs=(0x100002, 0x200000)) == EALIGN and clip(L, ptrs=(0x100002, 0x200000), dt=1) in NODEV
    assert clip(L, ptrs=(0x100000, None)) == EINVAL and clip(L, ptrs=(0x100000, None), sizes=(5, 0)) in NODEV
    assert clip(L, sizes=(5, -1)) == EINVAL and clip(L, sizes=(1 << 39, 1)) == EINVAL
    assert clip(L, bytes=639 * 8) == ENOSPACE and grad_norm(L, bytes=0) == ENOSPACE
    assert clip(L, given=1, work=None, bytes=0) in NODEV and clip(L, mx=float("inf")) in NODEV
    # the same twice, or overlapping: read in the norm, never written
    assert clip(L, ptrs=(0x100000, 0x100000)) == EINVAL and grad_norm(L, ptrs=(0x100000, 0x100000)) in NODEV
    assert clip(L, ptrs=(0x100000, 0x100000 + 3996)) == EINVAL and clip(L, ptrs=(0x200000, 0x100000)) in NODEV
    # elsewhere: apart from every gradient and from each other, or in the gradient's own place
    far = (0x300000, 0x400000)
    assert clip(L, out=far) in NODEV and clip(L, out=far, dt=1, od=0) in NODEV
    assert clip(L, out=(0x100000, 0x400000)) in NODEV and clip(L, out=(0x100000, 0x400000), dt=1, od=0) == EINVAL
    assert clip(L, ptrs=(0x100000, 0x100000), out=far) in NODEV  # read twice, written apart
    for out in ((0x300000, 0x300000), (0x200000, 0x100000), (0x100004, 0x400000), (None, 0x400000), (0x50000 - 400, 0x400000)):
        assert clip(L, out=out) == EINVAL, out
    assert clip(L, out=(0x300002, 0x400000)) == EALIGN
    assert L.demo_grad_workspace(0) == L.demo_grad_workspace(512) == 5120 and L.demo_grad_workspace(513) == 10240
    assert L.demo_grad_workspace(-1) == 0


def test_bindings_of_gradients_refuse_cpu_tensors():
    import decoupled_momentum_optimizer_gb300 as dm

    for call in (lambda: dm.grad_norm(torch.zeros(4)), lambda: dm.clip_grads([torch.zeros(4)], 1.0)):
        with pytest.raises(ValueError, match="no CPU path"):
            call()
