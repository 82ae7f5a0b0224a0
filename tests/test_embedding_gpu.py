"""Embedding lookup and its gradient on the GPU against their definitions in 64 bits.

A looked-up element is one float32 product and one rounding and is compared exactly; a gradient element is a
float32 sum in an order of its own, within one rounding of the sum of magnitudes per addition.
"""

import numpy as np
import pytest
import torch

import decoupled_momentum_optimizer_gb300 as dm
import model_ref as mr
from model_ref import DT, draw, f64

pytestmark = pytest.mark.gpu

IDX = {"i32": torch.int32, "i64": torch.int64}


def tokens(n, vocab, spread="zipf", padding=0.0, seed=60):
    gen = np.random.default_rng(seed)
    u = gen.random(n)
    if spread == "zipf":
        t = np.minimum((np.exp(u * np.log(vocab + 1)) - 1).astype(np.int64), vocab - 1)
    elif spread == "same":
        t = np.full(n, vocab // 2)
    elif spread == "distinct":
        t = gen.permutation(vocab)[np.arange(n) % vocab]
    else:
        t = (u * vocab).astype(np.int64)
    t[gen.random(n) < padding] = -1
    return torch.from_numpy(t)


def check_lookup(t, table, scale, odt, **kw):
    got = dm.embedding(t, table, scale=scale, dtype=DT[odt] if "out" not in kw else None, **kw)
    tt, tab = t.cpu().numpy(), f64(table).astype(np.float32)
    live = (tt >= 0) & (tt < tab.shape[0])
    want = np.zeros((*tt.shape, tab.shape[1]), dtype=np.float32)
    want[live] = tab[tt[live]] * np.float32(scale)
    assert got.shape == want.shape and np.array_equal(f64(got), mr.rounded(want, odt), equal_nan=True)
    return got


@pytest.mark.parametrize("tdt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("odt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,vocab,cols", [(1, 1, 1), (3, 7, 768), (1, 100, 2048), (40, 5, 63), (257, 1000, 8), (513, 300, 129),
                                          (2, 3, 8193)])
@pytest.mark.parametrize("idx", ["i32", "i64"])
def test_lookup(n, vocab, cols, tdt, odt, idx):
    t = tokens(n, vocab, "uniform", 0.2 if n > 10 else 0.0).to(IDX[idx]).cuda()
    check_lookup(t, draw(vocab, cols, tdt, 61), 27.7128, odt)


@pytest.mark.parametrize("tdt,odt", [("f32", "bf16"), ("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("pad,offset", [(3, 1), (8, 0), (0, 4), (8, 8)])
@pytest.mark.parametrize("cols", [64, 100, 765])
def test_lookup_strides(cols, pad, offset, tdt, odt):
    t = tokens(90, 40, "uniform", 0.1).cuda()
    out, fine = mr.guarded(90, cols, odt, offset, pad)
    got = check_lookup(t, draw(40, cols, tdt, 62, pad=pad, offset=offset), 1.0, odt, out=out)
    assert got is out and fine()


@pytest.mark.parametrize("idx", ["i32", "i64"])
def test_token_layouts(idx):
    """Any rows of consecutive tokens: transposed, sliced, repeated, a column, a scalar."""
    table = draw(50, 24, "f32", 63)
    t = tokens(60, 50, "uniform").to(IDX[idx]).cuda()
    dy = draw(60, 24, "f32", 64)
    for v in (t.view(5, 12)[:, 2:9], t.view(5, 12)[:, 3], t.view(3, 4, 5)[:, :, 1:4][:, :1], t[::3], t[:7].expand(4, 7),
              t[:1].expand(9), t.view(2, 5, 6)[:, 1:4], t[5], t.view(12, 5).t()[2], t[:0], t.view(5, 12)[:, :0],
              t.view(3, 4, 5)[:, ::2, 1:3]):  # 20 apart twice 10 apart: six rows of two
        got = check_lookup(v, table, 2.0, "f32")
        g = dy.reshape(-1)[:v.numel() * 24].view(*v.shape, 24)
        same = dm.embedding_grad(v.contiguous(), g, 50)
        assert got.shape == (*v.shape, 24) and torch.equal(dm.embedding_grad(v, g, 50), same)
    for v in (t.view(5, 12).t(), t.view(3, 4, 5)[:, :3, 1:3]):
        with pytest.raises(ValueError, match="rows of consecutive"):
            dm.embedding(v, table)


def test_tokens_outside_the_table():
    table = draw(20, 40, "f32", 65)
    t = torch.tensor([0, 19, 20, -1, -100, 1 << 40, -(1 << 40), (1 << 32) + 3, 5, -(1 << 63), (1 << 63) - 1]).cuda()
    got = check_lookup(t, table, 1.0, "f32")
    assert not bool(got[2:8].any()) and bool(got[8].any())
    dy = draw(11, 40, "f32", 66)
    grad = dm.embedding_grad(t, dy, 20)
    want = torch.zeros(20, 40, device="cuda")
    want[0], want[19], want[5] = dy[0], dy[1], dy[8]
    assert torch.equal(grad, want)
    assert dm.embedding(t, table[:0]).shape == (11, 40) and not bool(dm.embedding(t, table[:0]).any())
    assert dm.embedding_grad(t, dy, 0).shape == (0, 40)


def test_lookup_past_32_bits():
    table = torch.zeros((1 << 20) + 9, 4104, dtype=torch.bfloat16, device="cuda")
    table[-1] = 3.0
    t = torch.tensor([0, (1 << 20) + 8, 5, (1 << 20) + 8]).cuda()
    got = dm.embedding(t, table, scale=0.5)
    assert bool((got[1] == 1.5).all()) and bool((got[3] == 1.5).all()) and not bool(got[[0, 2]].any())
    n = (1 << 20) + 3
    t = torch.zeros(n, dtype=torch.int32, device="cuda")
    t[-1] = (1 << 20) + 8
    out = dm.embedding(t, table)
    assert bool((out[-1] == 3.0).all()) and not bool(out[:-1].any())


# ---- gradient ------------------------------------------------------------------------------------

def check_grad(t, dy, vocab, scale=1.0, add=False, out=None, seed=67):
    cols = dy.shape[-1]
    before = draw(vocab, cols, "f32", seed) if add else None
    if out is None:
        out = before.clone() if add else torch.full((vocab, cols), float("nan"), device="cuda")
    elif add:
        out.copy_(before)
    got = dm.embedding_grad(t, dy, scale=scale, out=out, add=add)
    assert got is out
    tt, d = t.cpu().numpy().reshape(-1).astype(np.int64), f64(dy).reshape(-1, cols)
    live = (tt >= 0) & (tt < vocab)
    scale = float(np.float32(scale))
    if vocab * cols <= 1 << 24:
        want, mag = np.zeros((vocab, cols)), np.zeros((vocab, cols))
        np.add.at(want, tt[live], d[live])
        np.add.at(mag, tt[live], np.abs(d[live]))
        rows = slice(None)
    else:  # the named rows alone; the others are compared below
        rows, inverse = np.unique(tt[live], return_inverse=True)
        want, mag = np.zeros((len(rows), cols)), np.zeros((len(rows), cols))
        np.add.at(want, inverse, d[live])
        np.add.at(mag, inverse, np.abs(d[live]))
    count = np.zeros(vocab)
    np.add.at(count, tt[live], 1)
    u = 2.0 ** -24
    # an addition a row, one more for each run of 65536 positions, the product with the scale
    tol = (count[rows][:, None] + 2 + len(tt) // 65536) * u * mag * abs(scale) + 2.0 ** -140
    want = want * scale
    if add:
        old = f64(before)[rows]
        want = want + old
        tol = tol + (1 + len(tt) // 65536) * u * (np.abs(old) + mag * abs(scale))
    g = f64(got) if isinstance(rows, slice) else f64(got[torch.from_numpy(rows).cuda()])
    assert (np.abs(g - want) <= tol).all(), float((np.abs(g - want) / tol).max())
    absent = torch.from_numpy(count == 0).cuda()
    if add:
        assert torch.equal(got[absent], before[absent])
    else:
        assert not bool(got[absent].any())
    return got


# one token, pieces of 8, 16 and 32 positions and their ends, clusters of one, two, four and eight CTAs, the
# longest sorted run and one more, three runs
COUNTS = [1, 2, 7, 8, 9, 31, 32, 33, 64, 100, 1000, 1023, 1024, 1025, 2048, 2049, 4097, 9000, 65536, 65537, 140000]


@pytest.mark.parametrize("n", COUNTS)
@pytest.mark.parametrize("spread", ["zipf", "same", "distinct", "uniform"])
@pytest.mark.parametrize("add", [False, True])
def test_grad_counts(n, spread, add):
    vocab, cols = 700 if n % 2 else 5000, 24 if n % 3 else 7
    check_grad(tokens(n, vocab, spread, 0.1 if n > 9 else 0.0).cuda(), draw(n, cols, "f32", 68), vocab, 3.0, add)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,vocab,cols", [(1, 1, 1), (5, 2, 9), (300, 40, 256), (300, 40, 264), (500, 100, 768), (3000, 50, 2048),
                                          (40, 3, 8200), (2000, 10, 127), (6000, 4000, 1024)])
@pytest.mark.parametrize("idx", ["i32", "i64"])
def test_grad_widths(n, vocab, cols, dtype, idx):
    t = tokens(n, vocab, "zipf", 0.1 if n > 9 else 0.0).to(IDX[idx]).cuda()
    check_grad(t, draw(n, cols, dtype, 69), vocab, 0.5, add=cols % 2 == 0)


@pytest.mark.parametrize("vocab", [1, 2, 255, 256, 511, 512, 513, 32128, 262143, 262144, (1 << 27) + 5, (1 << 28) + 5])
def test_grad_vocabularies(vocab):
    """Digits of one to nine bits, one to four passes; the first and the last token among them."""
    t = tokens(3000, vocab, "uniform", 0.05)
    t[5], t[77], t[2000], t[2001] = 0, vocab - 1, vocab - 1, vocab
    check_grad(t.cuda(), draw(3000, 1, "f32", 70), vocab)


@pytest.mark.parametrize("pad,offset", [(3, 1), (8, 0), (0, 4), (4, 4)])
@pytest.mark.parametrize("cols", [64, 100])
@pytest.mark.parametrize("add", [False, True])
def test_grad_strides(cols, pad, offset, add):
    out, fine = mr.guarded(90, cols, "f32", pad, offset)
    check_grad(tokens(500, 90, "zipf", 0.1).cuda(), draw(500, cols, "bf16", 71, pad=pad, offset=offset), 90, 2.0, add, out)
    assert fine()


def test_grad_sums_as_float32_does():
    """One token named 50000 times: not only within the worst case, but as good as the square root of it."""
    n, cols = 50000, 256
    dy = draw(n, cols, "bf16", 72)
    got = f64(dm.embedding_grad(torch.zeros(n, dtype=torch.int64, device="cuda"), dy, 1))[0]
    want = f64(dy).sum(0)
    assert np.linalg.norm(got - want) <= 4 * 2.0 ** -24 * np.sqrt(n) * np.linalg.norm(want)


@pytest.mark.parametrize("cols", [33, 128, 255, 300, 512, 767, 1000, 1024, 1033, 2056])
@pytest.mark.parametrize("n,pad", [(40, 0), (3000, 0), (3000, 4), (9000, 3), (20, 5)])
def test_grad_of_tables_longer_than_what_is_filled_first(n, pad, cols):
    """Rows without a token that the sums' kernel writes: alone, in runs, at the end; beside the rows, nothing."""
    vocab = (120 << 20) // (4 * cols) + 3
    t = torch.randint(0, vocab, (n,), generator=torch.Generator().manual_seed(74))
    t[: n // 2] = vocab - 1 - t[: n // 2] % 999  # a dense part at the end
    buf = torch.full((vocab, cols + pad), float("nan"), device="cuda")
    buf[:, cols:] = 5.0
    check_grad(t.cuda(), draw(n, cols, "bf16", 75), vocab, out=buf[:, :cols])
    assert bool((buf[:, cols:] == 5.0).all())


def test_grad_past_32_bits():
    vocab, cols = (1 << 20) + 9, 4104
    t = torch.tensor([3, vocab - 1, vocab - 1, 3, 3]).cuda()
    dy = draw(5, cols, "f32", 73)
    grad = torch.full((vocab, cols), 7.0, device="cuda")
    dm.embedding_grad(t, dy, out=grad)
    assert torch.equal(grad[-1], dy[1] + dy[2]) and torch.equal(grad[3], dy[0] + dy[3] + dy[4])
    assert not bool(grad[4:-1].any()) and not bool(grad[:3].any())
    n = (1 << 20) + 5
    big = torch.zeros(n, cols, dtype=torch.bfloat16, device="cuda")
    big[-2:] = 1.0
    t = torch.zeros(n, dtype=torch.int32, device="cuda")
    t[-1] = 2
    g = dm.embedding_grad(t, big, 3)
    assert bool((g[0] == 1).all()) and not bool(g[1].any()) and bool((g[2] == 1).all())


@pytest.mark.parametrize("n", [1, 5, 31, 32, 33])
@pytest.mark.parametrize("vocab,cols", [(1, 5), (31, 3), (700, 1), (700, 24), (5000, 768), (3, 2056), (300000, 7)])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("idx", ["i32", "i64"])
def test_few_positions(n, vocab, cols, add, idx):
    """Up to 32 are sorted by the warps that sum; one more takes the other kernels."""
    t = tokens(n, vocab, "zipf", 0.2 if n > 4 else 0.0).to(IDX[idx])
    if n > 4:
        t[1], t[3] = t[0], vocab - 1
    check_grad(t.cuda(), draw(n, cols, "bf16", 82, pad=cols % 2), vocab, 1.5, add)


def test_gradient_is_that_of_the_lookup():
    """sum(w * embedding) is linear in the table: a difference over a finite step is its derivative."""
    table, w = draw(30, 20, "f32", 74), draw(80, 20, "f32", 75)
    t = tokens(80, 30, "zipf", 0.2).cuda()
    grad = f64(dm.embedding_grad(t, w, 30, scale=1.5))

    def loss(tab):
        return (f64(dm.embedding(t, tab, scale=1.5)) * f64(w)).sum()

    for r, c in ((0, 0), (1, 19), (29, 3), (7, 11)):
        up = table.clone()
        up[r, c] += 2.0
        step = float(up[r, c].double() - table[r, c].double())
        bound = 2.0 ** -22 * float(w.double().abs().sum()) * (3 + float(table[r, c].abs()))
        assert abs((loss(up) - loss(table)) / step - grad[r, c]) <= bound


def test_non_finite_gradients_stay_with_their_tokens():
    t = torch.tensor([1, 2, 1, 3, 2, 1] * 20).cuda()
    dy = draw(120, 64, "f32", 76)
    want = dm.embedding_grad(t, dy, 5)
    dy[3, 5], dy[7, 6] = float("nan"), float("inf")
    got = dm.embedding_grad(t, dy, 5)
    bad = torch.zeros(5, 64, dtype=torch.bool, device="cuda")
    bad[t[3], 5], bad[t[7], 6] = True, True
    assert torch.equal(got[~bad], want[~bad]) and not bool(torch.isfinite(got[bad]).any())


def test_empty_calls():
    out = torch.ones(6, 8, device="cuda")
    none, dy = torch.zeros(0, dtype=torch.int64, device="cuda"), torch.zeros(0, 8, device="cuda")
    assert bool((dm.embedding_grad(none, dy, out=out, add=True) == 1).all())
    assert not bool(dm.embedding_grad(none, dy, out=out).any())
    assert dm.embedding_grad(none, dy[:, :0], 6).shape == (6, 0)
    assert dm.embedding(none, out).shape == (0, 8)
    padding = torch.full((40,), -1, device="cuda")
    assert not bool(dm.embedding_grad(padding, draw(40, 8, "f32", 77), 6).any())


def test_streams_repeats_and_graphs():
    """The same bits on another stream, from call to call, and from two graphs that share a workspace."""
    vocab, cols, n = 500, 768, 3000
    t, u = tokens(n, vocab, "zipf", 0.1).cuda(), tokens(n, vocab, "uniform", seed=61).cuda()
    dy, table = draw(n, cols, "bf16", 78), draw(vocab, cols, "f32", 79)
    want = dm.embedding(t, table, dtype=torch.bfloat16), dm.embedding_grad(t, dy, vocab)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dm.embedding(t, table, dtype=torch.bfloat16, stream=side), dm.embedding_grad(t, dy, vocab, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    work = torch.empty(dm.lib().demo_embedding_grad_workspace(n, cols), dtype=torch.uint8, device="cuda")
    a, b = t.clone(), u.clone()
    ga, gb = torch.empty(vocab, cols, device="cuda"), torch.empty(vocab, cols, device="cuda")
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        dm.embedding_grad(a, dy, out=ga, workspace=work)
    with torch.cuda.graph(second):
        dm.embedding_grad(b, dy, out=gb, workspace=work)
    for x, y in ((t, u), (u, t)):
        a.copy_(x), b.copy_(y)
        first.replay(), second.replay()
        assert torch.equal(ga, dm.embedding_grad(x, dy, vocab)) and torch.equal(gb, dm.embedding_grad(y, dy, vocab))


def test_refusals():
    table, t, dy = draw(20, 40, "f32", 80), tokens(10, 20).cuda(), draw(10, 40, "f32", 81)
    g = table.clone().requires_grad_()
    for call in (lambda: dm.embedding(t, g), lambda: dm.embedding_grad(t, dy.clone().requires_grad_(), 20),
                 lambda: dm.embedding_grad(t, dy, out=g)):
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    for err, call in ((TypeError, lambda: dm.embedding(t.short(), table)), (TypeError, lambda: dm.embedding([1], table)),
                      (ValueError, lambda: dm.embedding(t, table[0])), (ValueError, lambda: dm.embedding(t, table, out=dy[:9])),
                      (ValueError, lambda: dm.embedding(t, table.t())), (TypeError, lambda: dm.embedding(t, table, dtype=torch.int32)),
                      (dm.DemoError, lambda: dm.embedding(t, table, out=table[:10])),
                      (dm.DemoError, lambda: dm.embedding(t, table, scale=float("inf"))),
                      (ValueError, lambda: dm.embedding_grad(t, dy)), (ValueError, lambda: dm.embedding_grad(t, dy, 20, add=True)),
                      (ValueError, lambda: dm.embedding_grad(t[:9], dy, 20)), (ValueError, lambda: dm.embedding_grad(t, dy, 21, out=table)),
                      (TypeError, lambda: dm.embedding_grad(t, dy, out=table.half())),
                      (dm.DemoError, lambda: dm.embedding_grad(t.repeat(4), dy.repeat(4, 1), 20, workspace=small)),
                      (dm.DemoError, lambda: dm.embedding_grad(t, dy, out=dy))):
        with pytest.raises(err):
            call()
