"""Dropout, 8-bit quantization and its products on the GPU against their definitions in 64 bits.

Codes, scales and masks are compared exactly; computed values within bounds derived from the
number of float32 roundings (train_ref.product_tolerance, round_tolerance).
"""

import numpy as np
import pytest
import torch

import decoupled_momentum_optimizer_gb300 as dm
import train_ref as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def draw(rows, cols, dtype="f32", seed=0, std=1.0, pad=0, offset=0):
    """A [rows, cols] view whose rows are `pad` longer and start `offset` elements into the buffer."""
    gen = torch.Generator().manual_seed(seed)
    w = cols + pad
    x = torch.randn(rows * w + offset, generator=gen) * std
    x = x * torch.exp(torch.randn(rows * w + offset, generator=gen))
    return x.to(DT[dtype]).cuda()[offset:].view(rows, w)[:, :cols]


def f64(t):
    return t.double().cpu().numpy()


# ---- dropout -------------------------------------------------------------------------------------

SHAPES = [(1, 1), (1, 3), (3, 1), (1, 4), (5, 7), (1, 2048), (7, 768), (33, 765), (130, 63), (65, 132), (3, 4100),
          (2, 12), (1, 20), (257, 64)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("pad,offset,residual", [(0, 0, False), (0, 0, True), (3, 1, True), (8, 0, False), (4, 4, True)])
def test_dropout(rows, cols, dtype, pad, offset, residual):
    x = draw(rows, cols, dtype, 1, pad=pad, offset=offset)
    res = draw(rows, cols, dtype, 2, pad=pad, offset=offset) if residual else None
    got = dm.dropout(x, 0.3, seed=(1 << 63) + 5, step=7, site=11, residual=res)
    want, keep = ref.dropout(f64(x), 0.3, (1 << 63) + 5, 7, 11, f64(res) if residual else None)
    mag = np.abs(np.where(keep, f64(x) * ref.drop_scale(0.3), 0.0)) + (np.abs(f64(res)) if residual else 0.0)
    tol = 3 * 2.0 ** -24 * mag + ref.round_tolerance(want, dtype)
    assert (np.abs(f64(got) - want) <= tol).all()
    if not residual:
        assert ((f64(got) != 0) <= keep).all() and (f64(got)[keep & (np.abs(f64(x)) > 1e-4)] != 0).all()


@pytest.mark.parametrize("p", [0.0, 1.0, 2.0 ** -17, 1 - 2.0 ** -17, 0.5, 1.5 / 65536])
def test_dropout_probabilities(p):
    x = draw(40, 100, "f32", 3)
    got = f64(dm.dropout(x, p, seed=1, step=2))
    want, keep = ref.dropout(f64(x), p, 1, 2, 0)
    assert (np.abs(got - want) <= 2.0 ** -23 * np.abs(want)).all()
    assert ((got != 0) == keep).all()


@pytest.mark.parametrize("cols", [64, 65, 5])
def test_dropout_of_non_finite_values(cols):
    """A dropped infinity or NaN leaves 0 (or the residual), a kept one passes."""
    x = draw(16, cols, "f32", 4)
    x[::2] = float("nan")
    x[1::4] = float("inf")
    res = draw(16, cols, "f32", 5)
    keep = ref.keep_mask(16, cols, 0.5, 9, 9, 0)
    got, with_res = dm.dropout(x, 0.5, seed=9, step=9), dm.dropout(x, 0.5, seed=9, step=9, residual=res)
    assert (f64(got)[~keep] == 0).all() and (f64(with_res)[~keep] == f64(res)[~keep]).all()
    bad = ~np.isfinite(f64(x))
    assert (~np.isfinite(f64(got)[keep & bad])).all() and np.isfinite(f64(got)[keep & ~bad]).all()


def test_dropout_in_place_and_sliced():
    buf = draw(50, 130, "bf16", 6)
    want = dm.dropout(buf[:, :64], 0.2, seed=3, step=4, residual=buf[:, 64:128])
    left = buf.clone()
    dm.dropout(left[:, :64], 0.2, seed=3, step=4, residual=left[:, 64:128], out=left[:, :64])
    assert torch.equal(left[:, :64], want) and torch.equal(left[:, 64:], buf[:, 64:])
    other = buf.clone()  # the residual's place, a column slice of the buffer x is a slice of
    dm.dropout(other[:, :64], 0.2, seed=3, step=4, residual=other[:, 64:128], out=other[:, 64:128])
    assert torch.equal(other[:, 64:128], want) and torch.equal(other[:, :64], buf[:, :64])


def test_dropout_of_broadcast_rows_and_higher_dimensions():
    row = draw(1, 100, "f32", 7)
    got = dm.dropout(row.expand(6, 100), 0.4, seed=1, step=1)
    assert torch.equal(got, dm.dropout(row.repeat(6, 1), 0.4, seed=1, step=1))
    x = draw(30, 40, "f32", 8)
    assert torch.equal(dm.dropout(x.view(2, 15, 40), 0.4, seed=1, step=1).view(30, 40), dm.dropout(x, 0.4, seed=1, step=1))
    assert dm.dropout(x[:0], 0.4, seed=1, step=1).shape == (0, 40)
    assert dm.dropout(x[:, :0], 0.4, seed=1, step=1).shape == (30, 0)


def test_dropout_backward_against_differences():
    """d(sum(w * out))/dx is dropout(w): the map is linear, so a difference over a finite step is
    its derivative up to the roundings of the two evaluations."""
    x, w = draw(9, 31, "f32", 9), draw(9, 31, "f32", 10)
    kw = dict(seed=5, step=6, site=7)
    grad = f64(dm.dropout(w, 0.3, **kw))
    for i, j in [(0, 0), (3, 17), (8, 30), (4, 4), (7, 29)]:
        d = x.clone()
        d[i, j] += 2.0
        diff = (f64(dm.dropout(d, 0.3, **kw)) - f64(dm.dropout(x, 0.3, **kw))) * f64(w)
        assert abs(diff.sum() / 2.0 - grad[i, j]) <= 2.0 ** -20 * (1 + np.abs(f64(x)[i, j])) * (1 + abs(grad[i, j]))


def test_dropout_past_32_bits():
    """Positions and addresses past 2^32: the tail of a long bfloat16 tensor, against the mask."""
    cols, rows = 8192, (1 << 19) + 9
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    got = dm.dropout(x, 0.5, seed=2, step=3, out=x)
    T, G, key = ref.threshold(0.5), cols // 4, ref.sm(ref.sm(ref.sm(2) ^ 3) ^ 0)
    for r in (0, rows // 2, (1 << 19) - 1, 1 << 19, rows - 1):
        keep = [((ref.sm(key ^ (r * G + c // 4)) >> (16 * (c % 4))) & 0xFFFF) >= T for c in range(cols)]
        assert np.array_equal(f64(got[r]) != 0, np.array(keep))


# ---- quantization --------------------------------------------------------------------------------

def same_codes(q, want_codes, want_scales):
    codes, scales = f64(q.codes), f64(q.scales)
    assert np.array_equal(codes, want_codes, equal_nan=True)
    assert np.array_equal(scales[:, :q.shape[0]], want_scales)


def check_quantized(x, fmt, tiles, form="both", **kw):
    v = kw.pop("values", None)
    v = f64(x) if v is None else v
    q = dm.fp8_quantize(x, fmt=fmt, form=form, scales="tiles" if tiles else "rows", **kw)
    rows, cols = q if form == "both" else (q, q)
    if form != "cols":
        same_codes(rows, *ref.quantize(v, fmt, tiles))
    if form != "rows":
        same_codes(cols, *ref.quantize(np.ascontiguousarray(v.T), fmt, tiles))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,cols,pad,offset", [(1, 1, 0, 0), (1, 200, 0, 0), (3, 128, 0, 0), (130, 5, 3, 0),
                                                  (129, 260, 0, 0), (128, 256, 8, 0), (200, 131, 1, 1)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_quantize(rows, cols, pad, offset, dtype, fmt):
    x = draw(rows, cols, dtype, 20, pad=pad, offset=offset)
    check_quantized(x, fmt, False)


@pytest.mark.parametrize("form", ["rows", "cols", "both"])
@pytest.mark.parametrize("tiles", [False, True])
def test_quantize_forms(form, tiles):
    check_quantized(draw(150, 260, "f32", 21), "e4m3", tiles, form)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("tiles", [False, True])
def test_quantize_scales_at_their_edges(fmt, tiles):
    """Block maxima at, just above and just below a scale's limit, subnormal ones, zeros, the largest float."""
    top = ref.LIMITS[fmt][2]
    ups = [np.float32(top), np.nextafter(np.float32(top), np.float32(np.inf)), np.nextafter(np.float32(top), np.float32(0)),
           np.float32(1e-45), np.float32(2.0 ** -126), np.float32(0), np.finfo(np.float32).max, np.float32(2.0 ** -118)]
    x = draw(len(ups) * (128 if tiles else 1), 256, "f32", 22).cpu()
    per = x.shape[0] // len(ups)
    for i, u in enumerate(ups):
        part = x[i * per:(i + 1) * per]
        part.copy_((part / part.abs().max()).clamp(-1, 1).double().mul(float(u)).float().clamp(-float(u), float(u)))
        part[0, 7] = float(u)
        part[0, 200] = -float(u)
    check_quantized(x.cuda(), fmt, tiles, "rows")


def test_quantize_rounds_to_even():
    """Every midpoint between neighbouring codes of both formats, at scale 1."""
    for fmt, dt in (("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)):
        v = torch.arange(0, 128, dtype=torch.uint8).view(dt).float()
        v = v[torch.isfinite(v)]
        mid = (v[1:] + v[:-1]) / 2
        x = torch.zeros(2, 256)
        x[0, :len(mid)], x[1, :len(v)] = mid, v
        x[:, [0, 128]] = ref.LIMITS[fmt][2]
        check_quantized(x.cuda(), fmt, False, "rows")


@pytest.mark.parametrize("form", ["rows", "cols"])
@pytest.mark.parametrize("tiles", [False, True])
def test_quantize_non_finite(form, tiles):
    x = draw(140, 140, "f32", 23)
    x[3, 5], x[4, 6], x[139, 139] = float("nan"), float("inf"), float("-inf")
    x[7] = float("nan")  # a row of nothing finite
    check_quantized(x, "e4m3", tiles, form)
    check_quantized(x, "e5m2", tiles, form)


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("p", [0.3, 0.999])
def test_quantize_dropout_at_the_ends_of_the_range(p, tiles):
    """Blocks next to float32's smallest and largest values, whose products with dropout's factor
    underflow or overflow: v is what float32 makes of x * factor, not finite values are NaN codes."""
    x = draw(260, 256, "f32", 27)
    x[:20] *= 1e-44
    x[20:40] *= 1e-38
    x[40:60] *= 1e-33
    x[128:140] = x[128:140].clamp(-3, 3) * 1e38
    x[140, 5] = 3.3e38
    keep = ref.keep_mask(260, 256, p, 1, 2, 3)
    with np.errstate(over="ignore"):
        v = np.where(keep, x.cpu().numpy() * np.float32(ref.drop_scale(p)), np.float32(0))
    check_quantized(x, "e4m3", tiles, "both", values=v.astype(np.float64), p=p, seed=1, step=2, site=3)
    check_quantized(x, "e5m2", tiles, "both", values=v.astype(np.float64), p=p, seed=1, step=2, site=3)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("act", ["relu", "gate", "both"])
@pytest.mark.parametrize("p", [0.0, 0.25])
@pytest.mark.parametrize("cols,pad", [(260, 0), (131, 2)])
def test_quantize_with_activation_and_dropout(dtype, act, p, cols, pad):
    x, gate = draw(140, cols, dtype, 24, pad=pad), draw(140, cols, dtype, 25, pad=pad)
    gate[2, 3] = float("nan")
    x[2, 3] = float("inf")
    v = x.float().cpu().numpy()
    if act != "gate":
        v = np.maximum(v, np.float32(0))
    if p:
        keep = ref.keep_mask(140, cols, p, 8, 9, 10)
        v = np.where(keep, v * np.float32(ref.drop_scale(p)), np.float32(0))
    if act != "relu":
        v = np.where(f64(gate) > 0, v, np.float32(0))
    check_quantized(x, "e4m3", False, "both", values=v.astype(np.float64), relu=act != "gate",
                    gate=None if act == "relu" else gate, p=p, seed=8, step=9, site=10)


def test_quantize_empty_and_out():
    for shape in ((0, 5), (5, 0)):
        x = torch.zeros(shape, device="cuda")
        rows, cols = dm.fp8_quantize(x, form="both")
        assert rows.shape == shape and cols.shape == shape[::-1]
    x = draw(10, 20, "f32", 26)
    q = dm.Fp8Matrix.empty(10, 20)
    assert dm.fp8_quantize(x, out=q) is q
    assert torch.equal(q.codes.view(torch.uint8), dm.fp8_quantize(x).codes.view(torch.uint8))
    assert (f64(q.scales[:, 10:]) == 1).all()  # past the matrix up to the stride


def test_quantize_tall():
    """More row blocks than a grid's second dimension holds."""
    rows = 128 * 65536 + 5
    x = torch.zeros(rows, 4, dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.tensor([1.0, -2.0, 3.0, 448.0])
    q = dm.fp8_quantize(x, form="cols")
    assert f64(q.codes)[:, 128 * 65536 + 4].tolist() == [256.0, -256.0, 384.0, 448.0]
    assert f64(q.scales)[-1].tolist() == [2.0 ** -8, 2.0 ** -7, 2.0 ** -7, 1.0]


# ---- products ------------------------------------------------------------------------------------

def quantized(rows, k, fmt="e4m3", tiles=False, seed=0):
    q = dm.fp8_quantize(draw(rows, k, "f32", seed), fmt=fmt, scales="tiles" if tiles else "rows")
    return q, ref.values(f64(q.codes), f64(q.scales), k)


def check_product(m, n, k, a_fmt="e4m3", b_fmt="e4m3", tiles=False, out="f32", pad=0, offset=0, add=False):
    a, av = quantized(m, k, a_fmt, False, 30)
    b, bv = quantized(n, k, b_fmt, tiles, 31)
    want, total = ref.product(av, bv)
    dst = draw(m, n, out, 32, pad=pad, offset=offset)
    guard = dst._base.clone() if dst._base is not None else None
    if add:
        want, total = want + f64(dst), total + np.abs(f64(dst))
    got = dm.fp8_matmul(a, b, out=dst, add=add)
    assert got is dst
    err = np.abs(f64(got) - want)
    tol = ref.product_tolerance(total, k) + ref.round_tolerance(want, out) * (1 + 2.0 ** -8)
    assert (err <= tol).all(), float((err - tol).max())
    if k > 128 and out == "f32" and not add:  # the sums are as good as float32's, not only within bounds
        assert np.linalg.norm(err) <= 1e-6 * np.linalg.norm(total)
    return dst, guard


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 1, 128), (2, 3, 129), (128, 256, 128), (128, 256, 1024), (129, 257, 300),
                                   (5, 300, 515), (300, 5, 515), (256, 512, 2048), (260, 1000, 768), (513, 100, 4100), (700, 33, 9000),
                                   (2100, 1300, 700), (3000, 2000, 129), (5000, 450, 1024)])
@pytest.mark.parametrize("tiles", [False, True])
def test_matmul(m, n, k, tiles):
    check_product(m, n, k, tiles=tiles)


@pytest.mark.parametrize("a_fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("b_fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
def test_matmul_types(a_fmt, b_fmt, out):
    check_product(150, 300, 700, a_fmt, b_fmt, out=out)


@pytest.mark.parametrize("out,pad,offset", [("f32", 1, 0), ("f32", 4, 0), ("f32", 3, 0), ("f32", 0, 1), ("bf16", 3, 0), ("bf16", 7, 0),
                                            ("bf16", 8, 0), ("f16", 0, 2)])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("m,n", [(150, 300), (140, 64), (3, 33), (2500, 1377)])
def test_matmul_strides(out, pad, offset, add, m, n):
    if add and out != "f32":
        pytest.skip("add is float32's")
    dst, before = check_product(m, n, 300, out=out, pad=pad, offset=offset, add=add)
    flat, old = dst._base.reshape(-1), before.reshape(-1)
    inside = torch.zeros_like(flat, dtype=torch.bool)
    inside.as_strided(dst.shape, dst.stride(), dst.storage_offset()).fill_(True)
    assert torch.equal(flat[~inside], old[~inside])  # nothing around the result is written


def test_matmul_empty_sums():
    a, b = dm.Fp8Matrix.empty(5, 0), dm.Fp8Matrix.empty(7, 0)
    assert (f64(dm.fp8_matmul(a, b, dtype=torch.float32)) == 0).all()
    out = torch.ones(5, 7, device="cuda")
    assert (f64(dm.fp8_matmul(a, b, out=out, add=True)) == 1).all()
    assert dm.fp8_matmul(dm.Fp8Matrix.empty(0, 64), dm.Fp8Matrix.empty(7, 64)).shape == (0, 7)
    assert dm.fp8_matmul(dm.Fp8Matrix.empty(5, 64), dm.Fp8Matrix.empty(0, 64)).shape == (5, 0)


def test_matmul_any_power_of_two():
    """Scales that have nothing to do with the codes, and ones next to the ends of their range."""
    a, _ = quantized(130, 520, seed=33)
    b, _ = quantized(270, 520, seed=34)
    gen = torch.Generator().manual_seed(1)
    for q in (a, b):
        q.scales.copy_(torch.exp2(torch.randint(-12, 12, q.scales.shape, generator=gen).float()))
    a.scales[:, 3], b.scales[:, 5] = 2.0 ** -126, 2.0 ** 100
    av, bv = (ref.values(f64(q.codes), f64(q.scales), 520) for q in (a, b))
    want, total = ref.product(av, bv)
    got = f64(dm.fp8_matmul(a, b, dtype=torch.float32))
    over = np.abs(want) > float(np.finfo(np.float32).max)  # 2^100 * 2^11 * codes: past float32
    assert (got[over] == np.sign(want[over]) * np.inf).all()
    assert (np.abs(got - want)[~over] <= (ref.product_tolerance(total, 520) + 2.0 ** -126)[~over]).all()


def test_matmul_non_finite():
    """A NaN code spoils its row or column of the result and nothing else."""
    xa, xb = draw(140, 260, "f32", 35), draw(300, 260, "f32", 36)
    xa[7, 200], xb[290, 3] = float("inf"), float("nan")
    got = f64(dm.fp8_matmul(dm.fp8_quantize(xa), dm.fp8_quantize(xb), dtype=torch.float32))
    bad = np.zeros((140, 300), dtype=bool)
    bad[7], bad[:, 290] = True, True
    assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()


@pytest.mark.parametrize("m", [1, 7, 8, 9, 57, 64, 65, 104, 121, 127])
@pytest.mark.parametrize("n,k", [(500, 4200), (5000, 300)])
def test_matmul_of_few_rows(m, n, k):
    """Fewer rows than the tensor core multiplies: stages hold only those, and there are more of them."""
    check_product(m, n, k)


@pytest.mark.parametrize("m", [1, 9, 121])
def test_matmul_of_few_rows_next_to_non_finite_codes(m):
    """What the tensor core reads past a's rows (b's codes, a NaN among them) reaches no result."""
    xa, xb = draw(m, 1300, "f32", 43), draw(600, 1300, "f32", 44)
    xb[::2] = float("nan")
    got = f64(dm.fp8_matmul(dm.fp8_quantize(xa), dm.fp8_quantize(xb), dtype=torch.float32))
    assert np.isnan(got[:, ::2]).all() and np.isfinite(got[:, 1::2]).all()


@pytest.mark.parametrize("m,n,k", [(300, 500, 1500), (3000, 1500, 700)])
def test_matmul_repeats_to_the_bit_and_on_another_stream(m, n, k):
    a, _ = quantized(m, k, seed=37)
    b, _ = quantized(n, k, seed=38)
    first = dm.fp8_matmul(a, b, dtype=torch.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = dm.fp8_matmul(a, b, dtype=torch.float32)
    third = dm.fp8_matmul(a, b, dtype=torch.float32, stream=side)
    side.synchronize()
    assert torch.equal(first, again) and torch.equal(first, third)
    assert dm.device_fault() == 0


# ---- linear --------------------------------------------------------------------------------------

def check_linear(m, n, k, dtype="f32", out=None, fmt="e4m3", tiles=True, pad=0, offset=0, out_pad=0):
    x = draw(m, k, dtype, 40, pad=pad, offset=offset)
    w, wv = quantized(n, k, fmt, tiles, 41)
    codes, scales = ref.quantize(f64(x), "e4m3")
    want, total = ref.product(ref.values(codes, scales, k), wv)
    dst = draw(m, n, out or dtype, 42, pad=out_pad)
    before = dst._base.clone()
    got = dm.fp8_linear(x, w, out=dst)
    assert got is dst
    tol = ref.product_tolerance(total, k) + ref.round_tolerance(want, out or dtype) * (1 + 2.0 ** -8)
    err = np.abs(f64(got) - want)
    assert (err <= tol).all(), float((err - tol).max())
    outside = torch.ones_like(dst._base, dtype=torch.bool)
    outside.reshape(-1).as_strided(dst.shape, dst.stride(), dst.storage_offset()).fill_(False)
    assert torch.equal(dst._base[outside], before[outside])


@pytest.mark.parametrize("m", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 64, 65, 150])
@pytest.mark.parametrize("n,k", [(1, 1), (16, 128), (33, 300), (1000, 768), (257, 1411)])
def test_linear(m, n, k):
    check_linear(m, n, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("m", [1, 11, 70])
def test_linear_types(dtype, out, fmt, m):
    check_linear(m, 130, 515, dtype, out, fmt, tiles=fmt == "e4m3")


@pytest.mark.parametrize("dtype,pad,offset", [("f32", 1, 0), ("f32", 4, 4), ("bf16", 3, 1), ("bf16", 8, 8), ("bf16", 0, 1)])
@pytest.mark.parametrize("m", [1, 5, 20, 140])
@pytest.mark.parametrize("k", [300, 512])
def test_linear_strides(dtype, pad, offset, m, k):
    check_linear(m, 140, k, dtype, pad=pad, offset=offset, out_pad=3)


def test_linear_equals_quantize_then_matmul():
    """Few rows and many: the same codes, so results differ by their sums' roundings alone."""
    w, wv = quantized(500, 900, "e4m3", True, 43)
    for m in (1, 8, 30, 200):
        x = draw(m, 900, "bf16", 44)
        two = dm.fp8_matmul(dm.fp8_quantize(x), w, dtype=torch.float32)
        one = dm.fp8_linear(x, w, dtype=torch.float32)
        total = np.abs(f64(dm.fp8_quantize(x).dequantize())) @ np.abs(wv).T
        assert (np.abs(f64(one) - f64(two)) <= 2 * ref.product_tolerance(total, 900)).all()


@pytest.mark.parametrize("m", [2, 20, 130])
def test_linear_non_finite_and_empty(m):
    w, _ = quantized(100, 260, "e4m3", True, 45)
    x = draw(m, 260, "f32", 46)
    x[1, 5] = float("inf")
    got = f64(dm.fp8_linear(x, w))
    assert np.isnan(got[1]).all() and np.isfinite(np.delete(got, 1, 0)).all()
    assert dm.fp8_linear(x[:0], w).shape == (0, 100)
    empty = dm.Fp8Matrix.empty(100, 0)
    assert (f64(dm.fp8_linear(torch.empty(m, 0, device="cuda"), empty)) == 0).all()
    y = dm.fp8_linear(x.view(2, m // 2, 260), w, dtype=torch.bfloat16)
    assert y.shape == (2, m // 2, 100) and y.dtype == torch.bfloat16
    with pytest.raises(dm.DemoError):  # too small a workspace (or, for few rows, none is needed)
        dm.fp8_linear(draw(600, 260, "f32", 47), w, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))


def test_operators_in_a_graph():
    """The calls captured once and replayed on new contents give what they give outside."""
    x, w = draw(200, 300, "bf16", 50), draw(260, 300, "f32", 51)
    res = draw(200, 260, "bf16", 52)
    qw = dm.fp8_quantize(w, scales="tiles")

    def forward():
        q = dm.fp8_quantize(x, relu=True, p=0.2, seed=1, step=2)
        y = dm.fp8_matmul(q, qw)
        return dm.dropout(y, 0.1, seed=1, step=2, site=1, residual=res), dm.fp8_linear(x[:3], qw)

    forward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = forward()
    for seed in (53, 54):
        x.copy_(draw(200, 300, "bf16", seed))
        graph.replay()
        want = forward()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("call", ["pairs", "split", "linear"])
def test_a_load_that_never_completes_ends_in_the_fault_word(call):
    """The kernels' waits give up after their limit (2 s), every role stops, tensor memory is freed and
    the context stays usable: the same call gives the right result right after."""
    m, n, k = {"pairs": (2100, 1300, 700), "split": (200, 300, 2000), "linear": (3, 300, 2000)}[call]
    w, wv = quantized(n, k, "e4m3", True, 60)
    x = draw(m, k, "f32", 61)
    a = dm.fp8_quantize(x)
    run = (lambda: dm.fp8_linear(x, w)) if call == "linear" else (lambda: dm.fp8_matmul(a, w, dtype=torch.float32))
    want = run()
    assert dm.device_fault() == 0
    dm.test_stall_next_launch(0)
    run()
    assert dm.device_fault() == 1
    assert torch.equal(run(), want) and dm.device_fault() == 0


# ---- offsets past 32 bits ------------------------------------------------------------------------

def test_offsets_past_32_bits():
    """Codes, inputs and results of more than 2^32 elements: what is at their far ends."""
    rows, cols = (1 << 20) + 3, 4200  # 4.4e9 elements
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-130:] = draw(130, cols, "bf16", 70)
    x[:, -1] = 0.0
    x[-131:, -1] = torch.arange(1, 132).bfloat16().cuda()
    by_rows, by_cols = dm.fp8_quantize(x, form="both")
    want, scales = ref.quantize(f64(x[-2:]), "e4m3")
    assert np.array_equal(f64(by_rows.codes[-2:]), want) and np.array_equal(f64(by_rows.scales[:, rows - 2:rows]), scales)
    last = f64(x[rows // 128 * 128 - 256:, -1:])  # the last column, from a block's start
    want, scales = ref.quantize(np.ascontiguousarray(last.T), "e4m3")
    k0 = rows // 128 - 2
    assert np.array_equal(f64(by_cols.codes[-1:, k0 * 128:]), want)
    assert np.array_equal(f64(by_cols.scales[k0:, cols - 1]), scales[:, 0])
    del by_cols
    tokens = draw(3, cols, "bf16", 71)
    got = f64(dm.fp8_linear(tokens, by_rows, dtype=torch.float32))
    codes, sc = ref.quantize(f64(tokens), "e4m3")
    tail = dm.Fp8Matrix(by_rows.codes[-131:].contiguous(), torch.nn.functional.pad(by_rows.scales[:, rows - 131:rows], (0, 1)).contiguous(), cols)
    wv = f64(tail.dequantize())
    want, total = ref.product(ref.values(codes, sc, cols), wv)
    assert (np.abs(got[:, -131:] - want) <= ref.product_tolerance(total, cols)).all() and (got[:, :-131] == 0).all()
    tq = dm.fp8_quantize(tokens)
    want, total = ref.product(wv, f64(tq.dequantize()))
    got = f64(dm.fp8_matmul(by_rows, tq, dtype=torch.float32)[-131:])  # the long matrix as a
    assert (np.abs(got - want) <= ref.product_tolerance(total, cols)).all()
    del x, by_rows
    a, b = dm.fp8_quantize(draw(70001, 64, "f32", 72)), dm.fp8_quantize(draw(64000, 64, "f32", 73))
    out = dm.fp8_matmul(a, b)  # 4.5e9 results
    pick = [0, 33600, 70000]
    want, total = ref.product(f64(a.dequantize()[pick]), f64(b.dequantize()))
    tol = ref.product_tolerance(total, 64) + ref.round_tolerance(want, "bf16") * (1 + 2.0 ** -8)
    assert (np.abs(f64(out[pick]) - want) <= tol).all()
    odd = torch.empty(70001 * 64001, dtype=torch.bfloat16, device="cuda").view(70001, 64001)[:, :64000]
    dm.fp8_matmul(a, b, out=odd)  # rows that no bulk store can write
    assert torch.equal(odd[pick], out[pick]) and torch.equal(odd[-200:], out[-200:])


# ---- streams and shapes of the bindings ------------------------------------------------------------

def test_results_and_workspaces_belong_to_the_stream_they_are_used_on():
    """Calls queued behind a wait on another stream: what torch allocates meanwhile on this one may not
    take their buffers (a workspace is given back as soon as the call returns)."""
    w, _ = quantized(512, 1024, "e4m3", True, 80)
    x = draw(100, 1024, "bf16", 81)
    want = [dm.fp8_linear(x, w), dm.dropout(x, 0.5, seed=1, step=1), dm.fp8_matmul(dm.fp8_quantize(x), w)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)  # some tens of milliseconds
    got = [dm.fp8_linear(x, w, stream=side), dm.dropout(x, 0.5, seed=1, step=1, stream=side.cuda_stream)]
    got.append(dm.fp8_matmul(dm.fp8_quantize(x, stream=side), w, stream=side))
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in range(1024, 400 * 1024, 1024)]
    side.synchronize()
    assert len(junk) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_one_token_as_a_vector():
    w, _ = quantized(100, 260, "e4m3", True, 82)
    x = draw(2, 260, "f32", 83)
    assert torch.equal(dm.fp8_linear(x[0], w), dm.fp8_linear(x[:1], w)[0])
    assert dm.dropout(x[0], 0.1, seed=0, step=0).shape == (260,)


@pytest.mark.parametrize("row_blocks", [1, 2, 3, 4, 5, 6, 7, 9])
def test_linear_repeats_with_any_share_of_the_rows(row_blocks):
    """Every number of row blocks a CTA can own (the groups' rings of stages differ in length, and a last
    round may be short), called back to back: every result is the same to the bit and within bounds."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n, k = 16 * (sms * row_blocks - sms // 2), 2048
    w, wv = quantized(n, k, "e4m3", True, 90 + row_blocks)
    x = draw(3, k, "bf16", 91)
    codes, scales = ref.quantize(f64(x), "e4m3")
    want, total = ref.product(ref.values(codes, scales, k), wv)
    first = dm.fp8_linear(x, w, dtype=torch.float32)
    assert (np.abs(f64(first) - want) <= ref.product_tolerance(total, k)).all()
    outs = [torch.empty_like(first) for _ in range(50)]
    for _ in range(10):
        for out in outs:
            dm.fp8_linear(x, w, out=out)
        assert all(torch.equal(out, first) for out in outs)
    assert dm.device_fault() == 0


@pytest.mark.parametrize("m,k", [(1024, 4096), (256, 8192)])
def test_a_product_is_complete_when_the_next_encode_reads_it(m, k):
    """A gradient that a product writes last, encoded at once: the later replicas' encodes start before
    their predecessor's end, but not before the product's."""
    n, R = 2048, 3
    kw = dict(k=8, mode="demo", seed=4, step=2, wire="f32", beta=0.99, sign=True)
    ops = [(quantized(m, k, "e5m2", seed=95 + r)[0], quantized(n, k, seed=98 + r)[0]) for r in range(R)]
    runs = []
    for wait in (True, False, False, False):
        g = [torch.zeros(m * n, device="cuda") for _ in range(R)]
        mom = [torch.zeros(m * n, device="cuda") for _ in range(R)]
        pay = [dm.payload_buffers("demo", m * n, 8, step=2, wire="f32") for _ in range(R)]
        torch.cuda.synchronize()
        for r in range(R):
            dm.fp8_matmul(*ops[r], out=g[r].view(m, n), add=True)
        if wait:
            torch.cuda.synchronize()
        dm.encode_replicas(g, mom, [p[0] for p in pay], [p[1] for p in pay], **kw)
        runs.append(mom + [t for p in pay for t in p])
    for got in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got, runs[0]))
