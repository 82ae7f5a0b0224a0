"""The root-mean-square norm and its gradient on the GPU against their definitions in 64 bits.

The factors are within float32's rounding of the 64-bit value (2^-24, and the 2^-40 of the pairs' sum); given
them, the results, codes and scales are functions of two float32 products and are compared exactly.
"""

import numpy as np
import pytest
import torch

import decoupled_momentum_optimizer_gb300 as dm
import model_ref as mr
import train_ref as ref
from model_ref import DT, draw, f64

pytestmark = pytest.mark.gpu

EPS = 1e-6
RSTD = 2.0 ** -24 * (1 + 2.0 ** -15)

# one column, parts of an access, of a block and of a unit; a warp's registers full and one more; several warps
# and the widest row; few rows and many
SHAPES = [(1, 1), (3, 5), (7, 8), (5, 100), (9, 128), (2, 136), (6, 255), (40, 256), (11, 765), (4, 1023), (130, 1024),
          (1, 2048), (5, 2056), (3, 4100), (2, 8192), (33, 5000), (2, 16384), (3, 20001), (2, 32768), (3, 9001), (5, 12288), (1300, 200),
          (2500, 2048)]


def weight(cols, dtype, seed=50):
    return (1 + 0.3 * torch.randn(cols, generator=torch.Generator().manual_seed(seed))).to(DT[dtype]).cuda()


def check(x, w, dtype, residual=None, eps=EPS, form=None, fmt="e4m3", values=True, **kw):
    n = dm.rms_norm(x, w, eps=eps, residual=residual, form=form, fmt=fmt, values=values, save=True, **kw)
    s = f64(x)
    if residual is not None:
        s = mr.rounded(s.astype(np.float32) + f64(residual).astype(np.float32), dtype)
        assert np.array_equal(f64(n.total), s, equal_nan=True)
    r, want = f64(n.rstd), mr.norm_rstd(s, eps)
    assert np.array_equal(np.isnan(r), np.isnan(want))
    ok = ~np.isnan(want)
    assert (np.abs(r - want)[ok] <= RSTD * want[ok]).all()
    v = mr.norm_values(s, r, f64(w))
    if values:
        assert np.array_equal(f64(n.out), mr.rounded(v, dtype), equal_nan=True)
    if form is not None:
        forms = n.quantized if form == "both" else (n.quantized,)
        for name, q in zip(("rows", "cols") if form == "both" else (form,), forms):
            m = v if name == "rows" else np.ascontiguousarray(v.T)
            codes, scales = ref.quantize(m.astype(np.float64), fmt)
            assert np.array_equal(f64(q.codes), codes, equal_nan=True)
            assert np.array_equal(f64(q.scales)[:, :m.shape[0]], scales)
            assert (f64(q.scales)[:, m.shape[0]:] == 1).all()
    return n


@pytest.mark.parametrize("dtype,wdtype", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_values(rows, cols, dtype, wdtype):
    check(draw(rows, cols, dtype, 1), weight(cols, wdtype), dtype)
    check(draw(rows, cols, dtype, 1), weight(cols, wdtype), dtype, draw(rows, cols, dtype, 2, std=3.0))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad,offset", [(3, 1), (8, 0), (0, 4), (8, 8), (1, 0)])
@pytest.mark.parametrize("rows,cols", [(9, 256), (5, 765), (3, 2048), (2, 5000)])
def test_strides(rows, cols, dtype, pad, offset):
    x, res = draw(rows, cols, dtype, 3, pad=pad, offset=offset), draw(rows, cols, dtype, 4, pad=offset, offset=pad)
    out, fine = mr.guarded(rows, cols, dtype, pad, offset)
    total, fine2 = mr.guarded(rows, cols, dtype, offset, pad)
    n = check(x, weight(cols, "f32"), dtype, res, out=out, total=total)
    assert n.out is out and n.total is total and fine() and fine2()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("form", ["rows", "cols", "both"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (3, 128, 0), (5, 129, 0), (6, 136, 8), (133, 100, 3), (9, 765, 6),
                                           (2, 2048, 0), (260, 384, 0), (3, 4100, 4), (2, 16384 + 8, 0), (300, 3, 1), (77, 20, 0), (65, 40, 8)])
def test_forms(rows, cols, pad, dtype, form):
    x, res = draw(rows, cols, dtype, 5, pad=pad), draw(rows, cols, dtype, 6, pad=pad)
    check(x, weight(cols, "f32"), dtype, res, form=form, values=rows % 2 == 1)
    check(x, weight(cols, dtype), dtype, form=form, fmt="e5m2", values=rows % 2 == 0)


def test_fused_and_column_forms_agree():
    """The fused kernel's row codes, the tile kernel's and those of the quantizer on the float32 result."""
    x, w = draw(700, 1000, "f32", 7), weight(1000, "f32")
    one = dm.rms_norm(x, w, form="rows", values=True)
    rows, cols = dm.rms_norm(x, w, form="both", values=False).quantized
    q, qt = dm.fp8_quantize(one.out, form="both")
    for a, b in ((one.quantized, q), (rows, q), (cols, qt)):
        assert torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8)) and torch.equal(a.scales, b.scales)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [64, 100, 2048, 9000])
@pytest.mark.parametrize("eps", [1e-6, 1e-30, 1.0])
def test_far_values(dtype, cols, eps):
    """Rows whose squares leave float32's range, on either side; zeros; one large value among small ones."""
    x = draw(9, cols, dtype, 8)
    x[0] *= 1e-22
    x[1] *= 1e-37
    x[2] *= 1e19
    x[3] = (x[3] * 1e37).clamp(-3e38, 3e38)
    x[4] = 0.0
    x[5] *= 1e-12
    x[6, cols // 2] = 1e18
    x[7] *= 1e9
    check(x, weight(cols, "f32"), dtype, eps=eps, form="rows" if dtype == "f32" and eps == 1e-6 else None)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("cols", [100, 2048, 4100])
@pytest.mark.parametrize("form", [None, "rows", "both"])
def test_non_finite_rows_stay_among_themselves(dtype, cols, form):
    x = draw(8, cols, dtype, 9)
    x[1, 3], x[3, cols - 1], x[5, 0] = float("inf"), float("nan"), float("-inf")
    n = check(x, weight(cols, "f32"), dtype, form=form)
    assert f64(n.rstd)[1] == 0 and np.isnan(f64(n.rstd)[3])
    assert np.isfinite(f64(n.out)[[0, 2, 4, 6, 7]]).all()


def test_in_place():
    x, res, w = draw(30, 300, "bf16", 10), draw(30, 300, "bf16", 11), weight(300, "f32")
    want = dm.rms_norm(x, w, residual=res, save=True)
    a, b = x.clone(), res.clone()
    got = dm.rms_norm(a, w, residual=b, total=b, out=a, save=True)
    assert got.out is a and got.total is b
    assert all(torch.equal(p, q) for p, q in zip((got.out, got.total, got.rstd), (want.out, want.total, want.rstd)))
    c = x.clone()
    dm.rms_norm(c, w, out=c)
    assert torch.equal(c, dm.rms_norm(x, w).out)


def test_broadcast_rows_higher_dimensions_and_empty():
    x, w = draw(24, 64, "f32", 12), weight(64, "f32")
    want = dm.rms_norm(x, w, save=True)
    got = dm.rms_norm(x.view(2, 3, 4, 64), w, save=True)
    assert got.out.shape == (2, 3, 4, 64) and torch.equal(got.out.view(24, 64), want.out) and torch.equal(got.rstd, want.rstd)
    one = dm.rms_norm(x[:1].expand(5, 64), w, residual=x[:5])
    assert torch.equal(one.out, dm.rms_norm(x[:1].repeat(5, 1), w, residual=x[:5]).out)
    assert dm.rms_norm(x[:0], w, form="both").quantized[1].shape == (64, 0)
    assert dm.rms_norm(x[:, :0], w[:0], save=True).rstd.shape == (24,)
    n = dm.rms_norm(x, w, values=False, save=True)
    assert n.out is None and torch.equal(n.rstd, want.rstd) and n.total is x


def test_given_buffers():
    x, w = draw(70, 300, "bf16", 13), weight(300, "f32")
    q, qt = dm.Fp8Matrix.empty(70, 300), dm.Fp8Matrix.empty(300, 70)
    rstd = torch.empty(70, device="cuda")
    n = dm.rms_norm(x, w, form="both", quantized=(q, qt), rstd=rstd)
    assert n.quantized == (q, qt) and n.rstd is rstd
    m = dm.rms_norm(x, w, form="cols")
    assert m.rstd is None and torch.equal(m.quantized.codes.view(torch.uint8), qt.codes.view(torch.uint8))


def test_past_32_bits():
    rows, cols = (1 << 20) + 5, 4104
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    w = weight(cols, "f32")
    tail = draw(4, cols, "bf16", 14)
    x[-4:] = tail
    n = dm.rms_norm(x, w, form="rows", out=x, save=True)
    want = dm.rms_norm(tail, w, form="rows", save=True)
    assert torch.equal(x[-4:], want.out) and torch.equal(n.rstd[-4:], want.rstd) and not bool(x[:-4].any())
    assert torch.equal(n.quantized.codes[-4:].view(torch.uint8), want.quantized.codes.view(torch.uint8))
    dx, dw = dm.rms_norm_grad(x, x, w, n.rstd, out=x)
    a, b = dm.rms_norm_grad(want.out, want.out, w, want.rstd)
    assert torch.equal(dx[-4:], a) and torch.allclose(dw, b, rtol=1e-5, atol=1e-6 * float(b.abs().max()))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols,pad", [(1, 0), (3, 0), (3, 3), (20, 4), (64, 0), (100, 0), (128, 0), (130, 2)])
def test_many_short_rows(cols, pad, dtype):
    """Enough of them that a warp takes several at a time: every row is what it is in a call of a few rows, which the
    other tests compare with the formula.  The weight's gradient sums over all of them: a sum of n terms of random
    sign passes sums of the size of the result, each rounding 2^-24 of that, sqrt(n) of them together; eight times
    over."""
    lanes = 1
    while lanes < 32 and lanes * 4 < cols:
        lanes *= 2
    rows = 256 // lanes * 32 * torch.cuda.get_device_properties(0).multi_processor_count + 1037
    gen = torch.Generator(device="cuda").manual_seed(70)
    x, r = (torch.randn(rows, cols + pad, generator=gen, device="cuda").to(DT[dtype])[:, :cols] for _ in range(2))
    w = weight(cols, "f32")
    n = dm.rms_norm(x, w, residual=r, form="rows", save=True)
    dx, dw = dm.rms_norm_grad(x, n.total, w, n.rstd, past=r)
    for begin in (0, 4099, rows // 2 + 1, rows - 515):
        part = slice(begin, begin + 515)
        m = dm.rms_norm(x[part], w, residual=r[part], form="rows", save=True)
        for a, b in ((n.out, m.out), (n.total, m.total), (n.rstd, m.rstd)):
            assert torch.equal(a[part], b)
        assert torch.equal(n.quantized.codes[part].view(torch.uint8), m.quantized.codes.view(torch.uint8))
        assert torch.equal(n.quantized.scales[:, part], m.quantized.scales[:, :515])
        assert torch.equal(dx[part], dm.rms_norm_grad(x[part], m.total, w, m.rstd, past=r[part])[0])
    want = (x.double() * n.total.double() * n.rstd.double()[:, None]).sum(0)
    size = (x.double() * n.total.double() * n.rstd.double()[:, None]).square().sum(0).sqrt()
    assert bool(((dw.double() - want).abs() <= 8 * 2.0 ** -24 * rows ** 0.5 * size).all())


# ---- gradient ------------------------------------------------------------------------------------

def check_grad(rows, cols, dtype, wdtype="f32", past=True, add=False, pad=0, offset=0, std=1.0):
    s, dy = draw(rows, cols, dtype, 20, std=std, pad=pad, offset=offset), draw(rows, cols, dtype, 21, std=0.1)
    fl = draw(rows, cols, dtype, 22, std=0.1, pad=offset, offset=pad) if past else None
    w = weight(cols, wdtype)
    rstd = dm.rms_norm(s, w, save=True).rstd
    before = torch.randn(cols, generator=torch.Generator().manual_seed(23)).cuda() if add else None
    out, fine = mr.guarded(rows, cols, dtype, pad, offset)
    dx, dw = dm.rms_norm_grad(dy, s, w, rstd, past=fl, out=out, dweight=before.clone() if add else None, add=add)
    args = f64(dy), f64(s), f64(w), f64(rstd), None if fl is None else f64(fl)
    want, want_w, _, _ = mr.norm_grad(*args)
    tol, tol_w = mr.norm_grad_tolerance(*args, dtype, rows + 40)
    if add:
        want_w = want_w + f64(before)
        tol_w = tol_w + 2.0 ** -24 * np.abs(want_w)
    assert dx is out and fine()
    assert (np.abs(f64(dx) - want) <= tol).all(), float((np.abs(f64(dx) - want) / tol).max())
    assert (np.abs(f64(dw) - want_w) <= tol_w).all(), float((np.abs(f64(dw) - want_w) / tol_w).max())


@pytest.mark.parametrize("dtype,wdtype", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_grad(rows, cols, dtype, wdtype):
    check_grad(rows, cols, dtype, wdtype, past=rows % 2 == 0, add=cols % 2 == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad,offset", [(3, 1), (8, 0), (0, 4), (8, 8)])
@pytest.mark.parametrize("rows,cols", [(9, 256), (50, 765), (3, 2048), (300, 1000)])
def test_grad_strides(rows, cols, dtype, pad, offset):
    check_grad(rows, cols, dtype, pad=pad, offset=offset)


def test_grad_sums_over_many_rows_as_float32_does():
    """Not only within the worst case: the root mean square of n float32 roundings, four times over."""
    s, dy, w = draw(20000, 500, "bf16", 24), draw(20000, 500, "bf16", 25), weight(500, "f32")
    rstd = dm.rms_norm(s, w, save=True).rstd
    dw = f64(dm.rms_norm_grad(dy, s, w, rstd)[1])
    _, want, _, _ = mr.norm_grad(f64(dy), f64(s), f64(w), f64(rstd))
    assert np.linalg.norm(dw - want) <= 4 * 2.0 ** -24 * np.sqrt(20000) * np.linalg.norm(want)


def test_grad_formula_against_differences():
    """The 64-bit formula that the kernels are compared with, against central differences of the norm."""
    s, dy, w = (f64(draw(*a)) for a in ((5, 33, "f32", 26), (5, 33, "f32", 27), (1, 33, "f32", 28)))
    w = w[0]

    def loss(s, w):
        return (dy * s * mr.norm_rstd(s, EPS)[:, None] * w).sum()

    dx, dw, _, _ = mr.norm_grad(dy, s, w, mr.norm_rstd(s, EPS))
    for r, c in ((0, 0), (2, 17), (4, 32), (3, 5)):
        h = 1e-6
        up, down = s.copy(), s.copy()
        up[r, c] += h
        down[r, c] -= h
        assert abs((loss(up, w) - loss(down, w)) / (2 * h) - dx[r, c]) <= 1e-7 * np.abs(dx).max()
        up, down = w.copy(), w.copy()
        up[c] += h
        down[c] -= h
        assert abs((loss(s, up) - loss(s, down)) / (2 * h) - dw[c]) <= 1e-7 * np.abs(dw).max()


@pytest.mark.parametrize("place", ["dy", "total", "past"])
@pytest.mark.parametrize("dtype,cols", [("bf16", 2048), ("f32", 300)])
def test_grad_in_place(place, dtype, cols):
    t = dict(dy=draw(40, cols, dtype, 29), total=draw(40, cols, dtype, 30), past=draw(40, cols, dtype, 31))
    w = weight(cols, "f32")
    rstd = dm.rms_norm(t["total"], w, save=True).rstd
    want = dm.rms_norm_grad(t["dy"], t["total"], w, rstd, past=t["past"])
    got = dm.rms_norm_grad(t["dy"], t["total"], w, rstd, past=t["past"], out=t[place])
    assert got[0] is t[place] and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_grad_without_rows_and_without_weight():
    w, dw = weight(64, "f32"), torch.ones(64, device="cuda")
    x, r = torch.zeros(0, 64, device="cuda"), torch.zeros(0, device="cuda")
    assert not bool(dm.rms_norm_grad(x, x, w, r)[1].any())
    assert bool((dm.rms_norm_grad(x, x, w, r, dweight=dw, add=True)[1] == 1).all())
    s, dy = draw(40, 64, "f32", 32), draw(40, 64, "f32", 33)
    rstd = dm.rms_norm(s, w, save=True).rstd
    dx, none = dm.rms_norm_grad(dy, s, w, rstd, weight_grad=False)
    assert none is None and torch.equal(dx, dm.rms_norm_grad(dy, s, w, rstd)[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_grad_of_non_finite_rows_stays_among_them(dtype):
    s, dy, w = draw(50, 200, dtype, 34), draw(50, 200, dtype, 35), weight(200, "f32")
    rstd = dm.rms_norm(s, w, save=True).rstd
    want, _ = dm.rms_norm_grad(dy, s, w, rstd)
    s[7, 3], dy[9, 0] = float("nan"), float("inf")
    dx, dw = dm.rms_norm_grad(dy, s, w, dm.rms_norm(s, w, save=True).rstd)
    others = [i for i in range(50) if i not in (7, 9)]
    assert torch.equal(dx[others], want[others]) and not bool(torch.isfinite(dx[[7, 9]]).all())
    assert bool(torch.isnan(dw).all())  # a NaN row's factor spoils every column, as the formula says


# ---- streams, graphs, refusals -------------------------------------------------------------------

def test_streams_repeats_and_graphs():
    """The same bits on another stream, from call to call, and from a replayed graph on new contents."""
    x, res, dy = draw(300, 2048, "bf16", 36), draw(300, 2048, "bf16", 37), draw(300, 2048, "bf16", 38)
    w = weight(2048, "f32")

    def both(x, res, dy, stream=None):
        n = dm.rms_norm(x, w, residual=res, form="both", save=True, stream=stream)
        g = dm.rms_norm_grad(dy, n.total, w, n.rstd, past=dy, stream=stream)
        return [n.out, n.total, n.rstd, n.quantized[0].codes.view(torch.uint8), n.quantized[1].codes.view(torch.uint8), *g]

    want = both(x, res, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(x, res, dy, side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    a, b, c = x.clone(), res.clone(), dy.clone()
    both(a, b, c)
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = both(a, b, c)
    with torch.cuda.graph(other):
        second = both(b, a, c)
    for k in range(2):
        a.copy_(x if k else res), b.copy_(res if k else x)
        graph.replay()
        other.replay()
        now, swapped = both(a, b, c), both(b, a, c)
        assert all(torch.equal(p, q) for p, q in zip(first, now))
        assert all(torch.equal(p, q) for p, q in zip(second, swapped))


def test_refusals():
    x, w, dy = draw(8, 64, "bf16", 39), weight(64, "f32"), draw(8, 64, "bf16", 40)
    r = torch.ones(8, device="cuda")
    g = draw(8, 64, "bf16", 41).requires_grad_()
    with pytest.raises(ValueError, match="requires a gradient"):
        dm.rms_norm(g, w)
    with pytest.raises(ValueError, match="requires a gradient"):
        dm.rms_norm(x, w.clone().requires_grad_())
    with pytest.raises(ValueError, match="requires a gradient"):
        dm.rms_norm_grad(g, x, w, r)
    for err, call in ((TypeError, lambda: dm.rms_norm(x, w.half())), (ValueError, lambda: dm.rms_norm(x, w[:63])),
                      (ValueError, lambda: dm.rms_norm(x, w, total=x)), (ValueError, lambda: dm.rms_norm(x, w, form="tiles")),
                      (ValueError, lambda: dm.rms_norm(x.view(2, 4, 64), w, form="rows")),
                      (ValueError, lambda: dm.rms_norm(x, w, quantized=dm.Fp8Matrix.empty(8, 64))),
                      (ValueError, lambda: dm.rms_norm(x, w, form="rows", quantized=dm.Fp8Matrix.empty(64, 8))),
                      (ValueError, lambda: dm.rms_norm(x, w, fmt="e3m4")), (TypeError, lambda: dm.rms_norm(x, w, residual=w)),
                      (ValueError, lambda: dm.rms_norm(x, w, rstd=r[:7])), (ValueError, lambda: dm.rms_norm(x.t(), r.bfloat16())),
                      (dm.DemoError, lambda: dm.rms_norm(x, w, eps=0.0)), (dm.DemoError, lambda: dm.rms_norm(x, w, eps=float("nan"))),
                      (dm.DemoError, lambda: dm.rms_norm(x, w, out=x, form="cols")),
                      (dm.DemoError, lambda: dm.rms_norm(x, w, values=False)),
                      (ValueError, lambda: dm.rms_norm_grad(dy, x, w, r, add=True)),
                      (ValueError, lambda: dm.rms_norm_grad(dy, x, w, r[:7])),
                      (ValueError, lambda: dm.rms_norm_grad(dy, x, w, r, dweight=w.clone(), weight_grad=False)),
                      (ValueError, lambda: dm.rms_norm_grad(dy, x[:7], w, r)),
                      (ValueError, lambda: dm.rms_norm_grad(dy, x, w, r, workspace=r)),
                      (dm.DemoError, lambda: dm.rms_norm_grad(dy, x, w, r, workspace=torch.empty(100, dtype=torch.uint8, device="cuda"))),
                      (dm.DemoError, lambda: dm.rms_norm_grad(dy, x, w, r, dweight=w))):
        with pytest.raises(err):
            call()
    wide = torch.zeros(1, 32769, device="cuda")
    with pytest.raises(dm.DemoError):
        dm.rms_norm(wide, wide[0].clone())
