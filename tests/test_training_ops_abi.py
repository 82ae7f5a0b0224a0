"""The training operators' refusals, sizes and bindings without a GPU: every check runs before any
CUDA call, and valid arguments stop at the device check on a machine without one."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import train_ref as ref

OK, EINVAL, EALIGN, ENODEV, ENOTINIT, ENOSPACE = 0, -1, -2, -3, -5, -6
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "demo.h")


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


NODEV = (ENOTINIT, ENODEV)


def test_every_declared_operator_is_exported(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(demo_(?:dropout|fp8_[a-z_0-9]+))\s*\(", text))
    assert names == {"demo_dropout", "demo_fp8_bytes", "demo_fp8_quantize", "demo_fp8_matmul", "demo_fp8_linear",
                     "demo_fp8_linear_workspace"}
    for name in names:
        assert getattr(L, name).argtypes is not None


def dropout(L, **kw):
    a = dict(x=p(0x10000), ldx=100, res=None, ldr=100, out=p(0x90000), ldo=100, dtype=0, rows=10, cols=100, p=0.1, seed=0,
             step=0, site=0)
    a.update(kw)
    return L.demo_dropout(a["x"], a["ldx"], a["res"], a["ldr"], a["out"], a["ldo"], a["dtype"], a["rows"], a["cols"],
                          a["p"], a["seed"], a["step"], a["site"], None)


def test_dropout_refusals(L):
    assert dropout(L) in NODEV
    for bad in (dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(cols=-1), dict(p=-0.1), dict(p=1.1),
                dict(p=float("nan")), dict(x=None), dict(out=None), dict(ldo=99), dict(ldx=-1), dict(rows=1 << 40),
                dict(cols=1 << 40), dict(ldx=1 << 39)):
        assert dropout(L, **bad) == EINVAL, bad
    for bad in (dict(x=p(0x10002)), dict(out=p(0x90001)), dict(res=p(0x50002)), dict(x=p(0x10001), dtype=1)):
        assert dropout(L, **bad) == EALIGN, bad
    assert dropout(L, x=p(0x10002), dtype=1) in NODEV  # element alignment is enough
    assert dropout(L, rows=0) == OK and dropout(L, cols=0, x=None, out=None) == OK
    assert dropout(L, ldx=0) in NODEV and dropout(L, ldx=7) in NODEV  # an input's rows may repeat or overlap
    # in place is fine, a shifted overlap is not
    assert dropout(L, out=p(0x10000)) in NODEV and dropout(L, res=p(0x90000)) in NODEV
    assert dropout(L, out=p(0x10004)) == EINVAL and dropout(L, out=p(0x10000), ldo=101) == EINVAL
    assert dropout(L, res=p(0x90000 - 4)) == EINVAL
    # column slices of one buffer are apart; one column more is not
    cut = dict(x=p(0x10000), ldx=200, ldo=200)
    assert dropout(L, out=p(0x10000 + 400), **cut) in NODEV
    assert dropout(L, out=p(0x10000 + 396), **cut) == EINVAL and dropout(L, out=p(0x10000 + 404), **cut) == EINVAL
    assert dropout(L, x=p(0x10000 + 400), out=p(0x10000), ldx=200, ldo=200) in NODEV
    assert dropout(L, x=p(0x10000 + 404), out=p(0x10000), ldx=200, ldo=200) == EINVAL


def quantize(L, **kw):
    a = dict(x=p(0x100000), ldx=300, dtype=0, rows=200, cols=300, relu=0, gate=None, ldg=300, p=0.0, fmt=0, tiles=0,
             cr=p(0x1000000), sr=p(0x2000000), cc=p(0x3000000), sc=p(0x4000000))
    a.update(kw)
    return L.demo_fp8_quantize(a["x"], a["ldx"], a["dtype"], a["rows"], a["cols"], a["relu"], a["gate"], a["ldg"], a["p"],
                               0, 0, 0, a["fmt"], a["tiles"], a["cr"], a["sr"], a["cc"], a["sc"], None)


def test_quantize_refusals(L):
    assert quantize(L) in NODEV
    assert quantize(L, cc=None, sc=None) in NODEV and quantize(L, cr=None, sr=None) in NODEV
    for bad in (dict(dtype=3), dict(fmt=2), dict(rows=-1), dict(relu=2), dict(tiles=-1), dict(p=2.0), dict(x=None),
                dict(cr=None), dict(sc=None), dict(cr=None, sr=None, cc=None, sc=None), dict(ldx=-300),
                dict(rows=1 << 31), dict(rows=1 << 30, cols=1 << 30), dict(cr=p(0x100000)), dict(sr=p(0x1000000)),
                dict(cc=p(0x1000000 + 16)), dict(sc=p(0x100000 + 1024)), dict(gate=p(0x3000000))):
        assert quantize(L, **bad) == EINVAL, bad
    for bad in (dict(cr=p(0x1000008)), dict(sr=p(0x2000004)), dict(cc=p(0x3000001)), dict(sc=p(0x4000008)),
                dict(x=p(0x100002)), dict(gate=p(0x800001))):
        assert quantize(L, **bad) == EALIGN, bad
    assert quantize(L, rows=0) == OK and quantize(L, cols=0) == OK
    assert quantize(L, gate=p(0x100000)) in NODEV  # inputs may be shared


def matmul(L, **kw):
    a = dict(ac=p(0x1000000), asc=p(0x2000000), af=0, bc=p(0x3000000), bsc=p(0x4000000), bf=1, m=100, n=200, k=300,
             out=p(0x5000000), ldo=200, dtype=0, add=0)
    a.update(kw)
    return L.demo_fp8_matmul(a["ac"], a["asc"], a["af"], a["bc"], a["bsc"], a["bf"], a["m"], a["n"], a["k"], a["out"],
                             a["ldo"], a["dtype"], a["add"], None)


def test_matmul_refusals(L):
    assert matmul(L) in NODEV and matmul(L, add=1) in NODEV
    for bad in (dict(af=2), dict(bf=-1), dict(m=-1), dict(k=-1), dict(n=1 << 31), dict(m=1 << 30, n=1 << 30),
                dict(add=2), dict(add=1, dtype=1), dict(dtype=3), dict(ac=None), dict(bsc=None), dict(out=None),
                dict(ldo=199), dict(out=p(0x1000000)), dict(out=p(0x2000000)), dict(out=p(0x3000010)),
                dict(out=p(0x4000000 - 16))):
        assert matmul(L, **bad) == EINVAL, bad
    for bad in (dict(ac=p(0x1000008)), dict(asc=p(0x2000004)), dict(out=p(0x5000002)), dict(bc=p(0x3000001))):
        assert matmul(L, **bad) == EALIGN, bad
    assert matmul(L, m=0) == OK and matmul(L, n=0) == OK
    assert matmul(L, k=0, ac=None, asc=None, bc=None, bsc=None) in NODEV
    assert matmul(L, bc=p(0x1000000), bsc=p(0x2000000)) in NODEV  # inputs may be shared


def linear(L, **kw):
    a = dict(x=p(0x100000), ldx=300, dtype=1, wc=p(0x3000000), ws=p(0x4000000), wf=0, m=700, n=200, k=300,
             out=p(0x5000000), ldo=200, od=1, work=p(0x6000000), bytes=None)
    a.update(kw)
    if a["bytes"] is None:
        a["bytes"] = L.demo_fp8_linear_workspace(a["m"], a["n"], a["k"])
    return L.demo_fp8_linear(a["x"], a["ldx"], a["dtype"], a["wc"], a["ws"], a["wf"], a["m"], a["n"], a["k"],
                             a["out"], a["ldo"], a["od"], a["work"], a["bytes"], None)


def test_linear_refusals(L):
    assert linear(L) in NODEV
    for bad in (dict(dtype=3), dict(od=-1), dict(wf=2), dict(m=-1), dict(k=1 << 31), dict(x=None),
                dict(wc=None), dict(ws=None), dict(out=None), dict(work=None), dict(ldo=100), dict(ldx=-1),
                dict(out=p(0x100000)), dict(work=p(0x100000)), dict(work=p(0x5000000)), dict(work=p(0x3000000)),
                dict(m=1 << 30, n=1 << 20)):
        assert linear(L, **bad) == EINVAL, bad
    assert linear(L, bytes=L.demo_fp8_linear_workspace(700, 200, 300) - 1) == ENOSPACE
    for bad in (dict(x=p(0x100001)), dict(wc=p(0x3000008)), dict(work=p(0x6000004)), dict(out=p(0x5000001))):
        assert linear(L, **bad) == EALIGN, bad
    assert linear(L, m=0) == OK and linear(L, n=0) == OK
    assert linear(L, k=0, x=None, wc=None, ws=None, work=None) in NODEV


def test_sizes(L):
    sb = ctypes.c_size_t()
    for rows, k, codes, scales in ((1, 1, 128, 16), (5, 128, 640, 32), (5, 129, 1280, 64), (8, 0, 0, 0), (0, 8, 0, 0)):
        assert L.demo_fp8_bytes(rows, k, ctypes.byref(sb)) == codes and sb.value == scales
    assert L.demo_fp8_bytes(-1, 5, ctypes.byref(sb)) == 0 and sb.value == 0
    assert L.demo_fp8_bytes(5, 5, None) == 640
    assert L.demo_fp8_linear_workspace(0, 5, 5) == 0 and L.demo_fp8_linear_workspace(-1, 5, 5) == 0


def test_binding_refuses_cpu_tensors():
    import decoupled_momentum_optimizer_gb300 as dm

    x = torch.zeros(4, 8)
    codes, scales = torch.zeros(4, 128, dtype=torch.float8_e4m3fn), torch.ones(1, 4)
    for call in (lambda: dm.dropout(x, 0.1, seed=0, step=0), lambda: dm.fp8_quantize(x),
                 lambda: dm.fp8_linear(x, None), lambda: dm.Fp8Matrix(codes, scales, 8)):
        with pytest.raises(ValueError, match="no CPU path"):
            call()
    for codes2, scales2, k, err in ((codes.float(), scales, 8, TypeError), (codes, scales, 200, ValueError),
                                    (codes, torch.ones(1, 5), 8, ValueError), (codes[:, :64], scales, 8, ValueError)):
        with pytest.raises(err):
            dm.Fp8Matrix(codes2, scales2, k)
    with pytest.raises(AttributeError):
        dm.no_such_operator


def test_reference_mask_is_the_documented_hash():
    """The reference's mask against splitmix64's published outputs and the dropped share."""
    vec = open(os.path.join(os.path.dirname(__file__), "golden", "splitmix64_seed1234567.txt")).read().split()
    nums = [int(v) for v in vec if v.isdigit()]
    state = 1234567
    outs = []
    for _ in range(5):
        outs.append(ref.sm(state))
        state = (state + 0x9E3779B97F4A7C15) & ((1 << 64) - 1)
    assert all(o in nums for o in outs)
    keep = ref.keep_mask(100, 101, 0.3, 1, 2, 3)
    # 10100 draws at p = 0.3: four standard deviations
    assert abs(keep.mean() - 0.7) < 4 * np.sqrt(0.21 / keep.size)


def test_reference_code_is_the_nearest():
    """The reference's rounding against every representable value of both formats."""
    for fmt, dt in (("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)):
        v = torch.arange(0, 256, dtype=torch.int32).to(torch.uint8).view(dt).double().numpy()
        v = np.unique(v[np.isfinite(v)])
        for x in np.random.default_rng(0).normal(0, 30, 500):
            r = ref.round_code(x, fmt)
            assert r in v and abs(r - x) == np.abs(v - x).min()
