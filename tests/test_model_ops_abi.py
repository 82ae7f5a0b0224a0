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
