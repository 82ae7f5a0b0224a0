"""The gradients' norm and their clipping on the GPU against their definitions in 64 bits.

The norm: a float32 sum of at most eight squares, three joins, then float64: 11 roundings of a sum of
non-negative terms, halved by the root, and the rounding of the result.  Given the norm, a clipped element is
one float32 product and one rounding and is compared exactly.
"""

import numpy as np
import pytest
import torch

import decoupled_momentum_optimizer_gb300 as dm
import model_ref as mr
from model_ref import DT, f64

pytestmark = pytest.mark.gpu

NORM = (11 / 2 + 1) * 1.01 * 2.0 ** -24


def exact_norm(gs):
    return np.sqrt(sum(np.square(f64(g)).sum() for g in gs))


def check_norm(norm, want):
    got = float(norm.double())
    assert norm.dtype == torch.float32 and norm.shape == ()
    assert abs(got - want) <= NORM * want + 2.0 ** -150, (got, want)
    return np.float32(got)


def scaled(g, norm, max_norm, odt):
    f = np.float32(max_norm / np.float64(norm)) if max_norm < norm < np.inf else np.float32(1)
    return mr.rounded(f64(g).astype(np.float32) * f, odt)


def grads(sizes, dtype, gap=0, offset=0, std=1.0, seed=90):
    """Slices of one buffer, `gap` elements apart, from `offset` on; and the buffer."""
    gen = torch.Generator().manual_seed(seed)
    n = offset + sum(sizes) + gap * len(sizes) + 16
    buf = (torch.randn(n, generator=gen) * std).to(DT[dtype]).cuda()
    out, at = [], offset
    for size in sizes:
        out.append(buf[at:at + size])
        at += size + gap
    return out, buf


# nothing, one element, parts of an access, a chunk of either width and one more, several chunks
SIZES = [[1], [3], [4], [9], [0, 5, 0], [8191], [8192], [8193], [16384, 16385], [100000], [1, 2, 3, 4, 5, 6, 7, 8, 9],
         [768, 768 * 768, 1, 40000, 768], [64] * 511, [7] * 513, [33] * 1100, [3000000, 5],
         # around the longest list of one launch: 64 tensors, 64 chunks
         [9] * 64, [9] * 65, [8192] * 64, [8191] * 64, [8192] * 63 + [8193], [524288], [524289], [1048576], [1048577],
         [8192] * 65, [16384] * 63 + [0, 16384]]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gap,offset", [(0, 0), (1, 0), (5, 3), (8, 8)])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
def test_norm_and_clip(sizes, gap, offset, dtype):
    gs, buf = grads(sizes, dtype, gap, offset)
    want = exact_norm(gs)
    norm = check_norm(dm.grad_norm(gs), want)
    before = buf.clone()
    old, _ = grads(sizes, dtype, gap, offset)  # the same values
    for ratio in (2.0, 0.3):
        got = dm.clip_grads(gs, float(norm) * ratio)
        assert check_norm(got, want) == norm
        for g, o in zip(gs, old):
            assert np.array_equal(f64(g), scaled(o, norm, float(norm) * ratio, dtype))
        if ratio > 1:
            assert torch.equal(buf, before)  # nothing is written where nothing is clipped
    inside = torch.zeros_like(buf, dtype=torch.bool)
    for g in gs:
        inside[g.storage_offset():g.storage_offset() + g.numel()] = True
    assert torch.equal(buf[~inside], before[~inside])


@pytest.mark.parametrize("dtype,odt", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("gap,offset", [(0, 0), (1, 2), (8, 8), (3, 1)])
@pytest.mark.parametrize("ratio", [0.25, 3.0])
@pytest.mark.parametrize("longest", [70001, 1500001])  # one launch, two
def test_clip_into_other_tensors(dtype, odt, gap, offset, ratio, longest):
    sizes = [5000, 1, longest, 16, 9]
    gs, buf = grads(sizes, dtype, offset, gap)
    before = buf.clone()
    out, obuf = grads(sizes, odt, gap, offset, seed=91)
    around = obuf.clone()
    norm = check_norm(dm.clip_grads(gs, ratio * exact_norm(gs), out=out), exact_norm(gs))
    inside = torch.zeros_like(obuf, dtype=torch.bool)
    for g, o in zip(gs, out):
        assert np.array_equal(f64(o), scaled(g, norm, ratio * exact_norm(gs), odt))
        inside[o.storage_offset():o.storage_offset() + o.numel()] = True
    assert torch.equal(buf, before) and torch.equal(obuf[~inside], around[~inside])
    mixed = [gs[0], torch.empty_like(gs[1]), gs[2], torch.empty_like(gs[3]), torch.empty_like(gs[4])]
    if dtype == odt:
        dm.clip_grads(gs, ratio * exact_norm(gs), out=mixed)
        assert all(torch.equal(a, b) for a, b in zip(mixed, out))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("std", [1e-42, 1e-30, 1e-22, 1e-15, 1e18, 1e25, 3e35])
def test_all_of_the_range(dtype, std):
    """Squares past either end of float32; the clipped values too are the formula's."""
    gs, _ = grads([70000, 3, 900], dtype, 1, std=std)
    want = exact_norm(gs)
    norm = check_norm(dm.grad_norm(gs), want)
    old = [g.clone() for g in gs]
    dm.clip_grads(gs, float(norm) / 8)
    assert all(np.array_equal(f64(g), scaled(o, norm, float(norm) / 8, dtype)) for g, o in zip(gs, old))


def test_small_beside_large_and_zeros():
    g = torch.zeros(100000, device="cuda")
    g[5::8192] = 1e-30
    check_norm(dm.grad_norm(g), exact_norm([g]))
    g[77] = 1e30
    check_norm(dm.grad_norm(g), exact_norm([g]))
    z = torch.zeros(9000, device="cuda")
    assert float(dm.grad_norm([z, -z])) == 0.0
    assert float(dm.clip_grads(z, 0.0)) == 0.0 and not bool(z.any())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_norm_that_is_not_finite_scales_nothing(dtype, bad):
    gs, buf = grads([500, 20000, 7], dtype)
    gs[1][12345] = bad
    before, out = buf.clone(), [torch.empty_like(g) for g in gs]
    norm = float(dm.clip_grads(gs, 1e-3))
    assert norm == float("inf") if abs(bad) == float("inf") else norm != norm
    dm.clip_grads(gs, 1e-3, out=out)
    assert torch.equal(buf.view(torch.int16), before.view(torch.int16))
    assert all(torch.equal(a.view(torch.int16), b.contiguous().view(torch.int16)) for a, b in zip(out, gs))


def test_a_norm_past_float32():
    g = torch.full((1 << 20,), 3e38, device="cuda")
    assert float(dm.clip_grads(g, 1.0)) == float("inf") and bool((g == 3e38).all())


@pytest.mark.parametrize("given", [5.0, 0.5, float("inf"), float("nan"), 0.0])
def test_a_given_norm(given):
    gs, _ = grads([5000, 40], "f32")
    old = [g.clone() for g in gs]
    norm = torch.tensor(given, device="cuda")
    assert dm.clip_grads(gs, 1.0, norm=norm) is norm
    assert all(np.array_equal(f64(g), scaled(o, np.float32(given), 1.0, "f32")) for g, o in zip(gs, old))
    dm.clip_grads(gs, 0.0, norm=torch.ones((), device="cuda"))
    assert not any(bool(g.any()) for g in gs)


def test_shards_clipped_by_their_common_norm():
    gs, _ = grads([9000, 9000], "f32")
    old = [g.clone() for g in gs]
    whole = dm.grad_norm(gs)
    parts = torch.stack([dm.grad_norm(g) for g in gs])
    assert abs(float(parts.norm()) - float(whole)) <= 2.0 ** -21 * float(whole)
    for g in gs:
        dm.clip_grads(g, 1.0, norm=whole)
    assert all(np.array_equal(f64(g), scaled(o, np.float32(float(whole)), 1.0, "f32")) for g, o in zip(gs, old))


def test_norm_past_32_bits():
    g = torch.zeros((1 << 32) + 77, dtype=torch.bfloat16, device="cuda")
    g[1 << 31], g[-1], g[5] = 3.0, 4.0, 12.0
    assert float(dm.clip_grads(g, 6.5)) == 13.0
    assert g[-1] == 2.0 and g[1 << 31] == 1.5 and g[5] == 6.0


def test_the_same_gradient_twice():
    g = torch.ones(900, device="cuda")
    assert abs(float(dm.grad_norm([g, g])) - np.sqrt(1800.0)) <= 1e-5
    for call in (lambda: dm.clip_grads([g, g], 1.0), lambda: dm.clip_grads([g[:500], g[499:]], 1.0),
                 lambda: dm.clip_grads([g[:400], g[500:]], 1.0, out=[g[100:500], g[500:]]),
                 lambda: dm.clip_grads(g, 1.0, norm=g[5]), lambda: dm.grad_norm(g, out=g[:1])):
        with pytest.raises(dm.DemoError):
            call()
    assert bool((g == 1).all())


@pytest.mark.parametrize("sizes", [[768, 768 * 768, 40000, 5], [768, 1500 * 1024, 40000, 5]], ids=["one launch", "two"])
def test_streams_repeats_and_graphs(sizes):
    gs, buf = grads(sizes, "bf16", 3)
    fresh = buf.clone()
    want = dm.grad_norm(gs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dm.grad_norm(gs, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    work = torch.empty(dm.lib().demo_grad_workspace(4), dtype=torch.uint8, device="cuda")
    dm.clip_grads(gs, 1.0, workspace=work)
    clipped = buf.clone()
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        a = dm.clip_grads(gs, 1.0, workspace=work)
    with torch.cuda.graph(second):
        b = dm.grad_norm(gs[1:], workspace=work)
    for k in (1.0, 2.0):
        buf.copy_(fresh * k)
        second.replay(), first.replay()
        assert torch.equal(b, dm.grad_norm([(g * 1) for g in grads(sizes, "bf16", 3)[0][1:]]) * k)
        assert torch.equal(a, want * k)
        if k == 1.0:
            assert torch.equal(buf, torch.where(torch.ones_like(buf, dtype=torch.bool), clipped, buf))


def test_refusals():
    g = torch.ones(10, device="cuda")
    r = torch.ones(10, device="cuda", requires_grad=True)
    for err, call in ((ValueError, lambda: dm.grad_norm([])), (TypeError, lambda: dm.grad_norm(g.double())),
                      (TypeError, lambda: dm.grad_norm([g, g.half()])), (ValueError, lambda: dm.grad_norm([g, g.cpu()])),
                      (ValueError, lambda: dm.grad_norm(torch.ones(4, 4, device="cuda").t()[:, :2])),
                      (ValueError, lambda: dm.grad_norm(r)), (ValueError, lambda: dm.clip_grads([g, r], 1.0)),
                      (ValueError, lambda: dm.clip_grads(g, 1.0, out=torch.ones(9, device="cuda"))),
                      (ValueError, lambda: dm.clip_grads([g, g + 1], 1.0, out=[torch.ones(10, device="cuda")])),
                      (dm.DemoError, lambda: dm.clip_grads(g, 1.0, out=g.half())),
                      (dm.DemoError, lambda: dm.clip_grads(g, -1.0)), (dm.DemoError, lambda: dm.clip_grads(g, float("nan"))),
                      (ValueError, lambda: dm.clip_grads(g, 1.0, norm=g)),
                      (ValueError, lambda: dm.clip_grads(g, 1.0, norm=torch.ones((), dtype=torch.float64, device="cuda"))),
                      (ValueError, lambda: dm.grad_norm(g, workspace=g)),
                      (dm.DemoError, lambda: dm.grad_norm(g, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")))):
        with pytest.raises(err):
            call()
    with torch.no_grad():
        dm.clip_grads(r, 1.0)
    assert bool((g == 1).all()) and float(dm.grad_norm(r.detach())) < 1.001
