"""What the operators between the products and the optimizer step compute, and the calls that are timed.

  norm        root-mean-square norm of a row, with the residual's addition before it, into 16 or 32 bits
              and / or into 8-bit codes with a scale for each block of 128 (by rows, columns or both)
  norm_grad   its gradient: of the summed row (with what flows past the norm added) and of the weight
  embed       rows of a table by token, scaled
  embed_grad  its gradient: the rows of equal tokens summed, into a float32 table or added to it
  clip        the norm over all gradients of a model, and the gradients scaled to a largest norm

``run`` computes them with elementary torch operations in 32 bits (the mean square and the global sum of
squares in 64), or, where ``own`` is true, with this package's calls.  ``exact`` restates each definition
in 64 bits.

Norm of a row x [cols] with weight w: s = x + residual, rounded to x's type; rstd is the float32 nearest
to 1 / sqrt(mean(s^2) + eps); v = (s rstd) w, two float32 products.  The result is v rounded to x's type;
the 8-bit form is taken from v itself: kb = ceil(cols / 128) blocks along a row, the scale of a block the
smallest power of two s >= 2^-126 with amax <= 448 s (1 for zeros), the codes v / s rounded to nearest
even, [rows, 128 kb], zero past cols; scales float32 [kb, rows].  With dy the result's gradient, xh = s rstd
and c = mean(dy w xh): ds = rstd (dy w - xh c) + what flows past, dw = sum over rows of dy xh.

Tokens outside [0, vocab) give rows of zeros and no gradient.

Clipping leaves gradients whose norm is at most max_norm as they are, and multiplies others by
max_norm / norm.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 128
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6


# ---- cases ---------------------------------------------------------------------------------------

def listed():
    return [
        # one token between two layers of a width-2048 model that answers: nothing but latency
        dict(name="norm-token", op="norm", rows=1, cols=2048, dtype="bf16", weight="f32", residual=True, pad=0,
             form="none", values=True),
        # the norm before a feed-forward layer in training: its product and its weight gradient take 8 bits
        dict(name="norm-both", op="norm", rows=16384, cols=2048, dtype="bf16", weight="f32", residual=True, pad=0,
             form="both", values=False),
        # eight images' tokens at an odd width in a wider buffer, float32: the result and its 8-bit form
        dict(name="norm-odd-f32", op="norm", rows=8 * 197, cols=765, dtype="f32", weight="f32", residual=False, pad=6,
             form="rows", values=True),
        # a full training batch with the gradient that flows past the norm, the weight's added to the flat gradient
        dict(name="norm-grad-large", op="norm_grad", rows=32768, cols=2048, dtype="bf16", weight="f32", past=True,
             pad=0, add=True),
        # the same backward for the eight images
        dict(name="norm-grad-odd-f32", op="norm_grad", rows=8 * 197, cols=765, dtype="f32", weight="f32", past=False,
             pad=6, add=False),
        # three words entering a width-768 model
        dict(name="embed-few", op="embed", n=3, vocab=32128, cols=768, table="f32", dtype="bf16", index="i64",
             scale=27.712812921102035, spread="zipf", padding=0.0),
        # a full batch of text from the float32 shard of a width-2048 model
        dict(name="embed-batch", op="embed", n=16384, vocab=100352, cols=2048, table="f32", dtype="bf16", index="i64",
             scale=1.0, spread="zipf", padding=0.0),
        # its gradient, added to the flat gradient that the output layer of a tied table has written
        dict(name="embed-grad-tied", op="embed_grad", n=16384, vocab=100352, cols=2048, dtype="bf16", index="i64",
             scale=1.0, spread="zipf", padding=0.0, add=True),
        # short sentences, a fifth of the batch padding, of a width-768 model: every row of the gradient is written
        dict(name="embed-grad-sparse", op="embed_grad", n=4096, vocab=32128, cols=768, dtype="bf16", index="i32",
             scale=27.712812921102035, spread="zipf", padding=0.2, add=False),
        # the gradients of a two-layer probe: nothing but latency
        dict(name="norm-of-few", op="clip", layers=2, width=64, ff=160, vocab=500, dtype="f32", odd=False, ratio=0.0,
             out=False),
        # a width-768 model of 24 layers, each weight a tensor of its own, clipped to a tenth
        dict(name="clip-model", op="clip", layers=24, width=768, ff=2048, vocab=32128, dtype="f32", odd=False,
             ratio=0.1, out=True),
        # one replica's flat bfloat16 gradient of 2^27 parameters in a step that needs no clipping
        dict(name="clip-flat-unclipped", op="clip", layers=0, width=2048, ff=0, vocab=65536, dtype="bf16", odd=False,
             ratio=2.0, out=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size over the logarithm of the range; half of them whole multiples of 16."""
    v = _log(rng, lo, hi)
    return max(lo, v // 16 * 16) if rng.random() < 0.5 and v >= 16 else v


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "norm_grad", "embed", "embed_grad", "embed_grad", "clip", "clip"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op in ("norm", "norm_grad"):
        cols = _size(rng, 1, 16384)
        c = dict(op=op, rows=_log(rng, 1, max(1, 2 ** 25 // cols)), cols=cols, dtype=dtype,
                 weight=rng.choice(["f32", dtype]), pad=rng.choice([0, 0, 3, 8]))
        if op == "norm":
            form = rng.choice(["none", "rows", "cols", "both"])
            return dict(c, residual=rng.random() < 0.6, form=form, values=form == "none" or rng.random() < 0.5)
        return dict(c, past=rng.random() < 0.6, add=rng.random() < 0.5)
    if op in ("embed", "embed_grad"):
        cols = _size(rng, 1, 8192)
        n, vocab = _log(rng, 1, max(1, min(2 ** 17, 2 ** 25 // cols))), _log(rng, 1, max(1, min(2 ** 18, 2 ** 27 // cols)))
        c = dict(op=op, n=n, vocab=vocab, cols=cols, dtype=dtype, index=rng.choice(["i32", "i64"]),
                 scale=rng.choice([1.0, math.sqrt(cols)]), spread=rng.choice(["zipf", "uniform", "few"]),
                 padding=rng.choice([0.0, 0.0, 0.1, 0.5]))
        return dict(c, table=rng.choice(["f32", "f32", dtype])) if op == "embed" else dict(c, add=rng.random() < 0.5)
    width = _size(rng, 8, 2048)
    layers = _log(rng, 1, max(1, min(48, 2 ** 26 // (8 * width * width))))
    ratio = rng.choice([0.0, 0.05, 0.7, 1.5])
    return dict(op=op, layers=layers, width=width, ff=_log(rng, width, 2 * width), vocab=_log(rng, 2, 32768), dtype=dtype,
                odd=rng.random() < 0.4, ratio=ratio, out=0.0 < ratio < 1.0)


def _numels(case):
    """Elements of each gradient: the table, then four projections, two of the feed-forward and two norms a layer."""
    w, ff = case["width"], case["ff"]
    return [case["vocab"] * w] + case["layers"] * ([w * w] * 4 + [w * ff] * 2 + [w] * 2)


def work(case):
    op = case["op"]
    if op == "clip":
        e = sum(_numels(case))
        b = e * SIZES[case["dtype"]] * (2 if case["out"] else 1)
        return {"bytes": b + 4, "flops": 2 * e + (e if case["out"] else 0)}
    size, cols = SIZES[case["dtype"]], case["cols"]
    if op == "norm":
        rows = case["rows"]
        e = rows * cols
        b = e * size * (1 + 2 * case["residual"] + case["values"]) + cols * SIZES[case["weight"]]
        if case["form"] in ("rows", "both"):
            b += rows * (_pad(cols) + 4 * (_pad(cols) // BLOCK))
        if case["form"] in ("cols", "both"):
            b += cols * (_pad(rows) + 4 * (_pad(rows) // BLOCK))
        return {"bytes": b + 4 * rows, "flops": 5 * e}
    if op == "norm_grad":
        rows = case["rows"]
        return {"bytes": rows * cols * size * (3 + case["past"]) + 4 * rows
                + cols * (SIZES[case["weight"]] + (8 if case["add"] else 4)), "flops": 9 * rows * cols}
    n, vocab, index = case["n"], case["vocab"], 4 if case["index"] == "i32" else 8
    live = n * (1 - case["padding"])
    distinct = {"few": min(vocab, 3, live), "uniform": vocab * (1 - math.exp(-live / vocab)),
                "zipf": sum(1 - math.exp(-live * math.log1p(1 / (k + 1)) / math.log(vocab + 1))
                            for k in range(vocab))}[case["spread"]]
    if op == "embed":
        return {"bytes": int(n * index + distinct * cols * SIZES[case["table"]] + n * cols * size), "flops": n * cols}
    rows = 2 * distinct if case["add"] else vocab
    return {"bytes": int(n * index + live * cols * size + rows * cols * 4), "flops": int(live * cols)}


def _pad(k):
    return (k + BLOCK - 1) // BLOCK * BLOCK


# ---- inputs --------------------------------------------------------------------------------------

def _strided(gen, rows, cols, pad, dtype, std):
    """Values with a spread of channel sizes, in a buffer whose rows are `pad` elements longer."""
    x = torch.randn(rows, cols + pad, generator=gen, device="cuda") * std
    x *= torch.exp(0.5 * torch.randn(cols + pad, generator=gen, device="cuda"))
    return x.to(dtype)[:, :cols]


def _tokens(gen, case):
    n, vocab = case["n"], case["vocab"]
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    if case["spread"] == "zipf":  # token k about as often as 1 / (k + 1), as words are
        t = torch.exp(u * math.log(vocab + 1)) - 1
    else:
        t = u * (vocab if case["spread"] == "uniform" else min(vocab, 3))
    t = t.long().clamp(0, vocab - 1)
    padding = torch.rand(n, generator=gen, device="cuda") < case["padding"]
    return torch.where(padding, torch.full_like(t, -1), t).to(torch.int32 if case["index"] == "i32" else torch.int64)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("norm", "norm_grad"):
        dt, rows, cols = DTYPES[case["dtype"]], case["rows"], case["cols"]
        s["w"] = (1 + 0.2 * torch.randn(cols, generator=gen, device="cuda")).to(DTYPES[case["weight"]])
        s["x"] = _strided(gen, rows, cols, case["pad"], dt, 1.0)
        if op == "norm":
            if case["residual"]:
                s["residual"] = _strided(gen, rows, cols, case["pad"], dt, 2.0)
            return s
        s["rstd"] = s["x"].double().square().mean(1).add(EPS).rsqrt().float()  # as the forward pass left it
        s["dy"] = _strided(gen, rows, cols, case["pad"], dt, 1e-2)
        if case["past"]:
            s["past"] = _strided(gen, rows, cols, case["pad"], dt, 1e-2)
        if case["add"]:
            s["dw"] = torch.randn(cols, generator=gen, device="cuda")
        return s
    if op in ("embed", "embed_grad"):
        s["tokens"] = _tokens(gen, case)
        if op == "embed":
            s["table"] = (torch.randn(case["vocab"], case["cols"], generator=gen, device="cuda") * 2e-2).to(
                DTYPES[case["table"]])
            return s
        s["dy"] = _strided(gen, case["n"], case["cols"], 0, DTYPES[case["dtype"]], 1e-2)
        if case["add"]:
            s["grad"] = torch.randn(case["vocab"], case["cols"], generator=gen, device="cuda") * 1e-3
        return s
    # Every gradient is a slice of one buffer, 32 elements aligned, or one element apart.
    numels, offsets, at = _numels(case), [], 0
    for n in numels:
        offsets.append(at)
        at += n + 1 if case["odd"] else (n + 31) // 32 * 32
    flat = (torch.randn(at, generator=gen, device="cuda") * 1e-3).to(DTYPES[case["dtype"]])
    s["gs"] = [flat[o:o + n] for o, n in zip(offsets, numels)]
    if case["out"]:
        s["flat"] = torch.zeros_like(flat)
        s["outs"] = [s["flat"][o:o + n] for o, n in zip(offsets, numels)]
    else:
        s["flat"] = flat
    s["max_norm"] = case["ratio"] * 1e-3 * math.sqrt(sum(numels))
    return s


# ---- plain form ----------------------------------------------------------------------------------

def _pow2(e):
    return ((e + 127) << 23).view(torch.float32)


def _quantized(x):
    """Codes and scales of a float32 matrix by rows."""
    rows, k = x.shape
    kp = _pad(k)
    x = torch.nn.functional.pad(x, (0, kp - k)).reshape(rows, kp // BLOCK, BLOCK)
    mant, e = torch.frexp(x.abs().amax(2))
    e = torch.where(mant > 0, (e - 9 + (mant > 0.875)).clamp(min=-126), torch.zeros_like(e)).to(torch.int32)
    codes = (x * _pow2(-e).unsqueeze(2)).reshape(rows, kp).to(torch.float8_e4m3fn)
    return [codes, _pow2(e).t().contiguous()]


def run(state):
    s, case = state, state["case"]
    if own:
        return _run_own(s, case, case["op"])
    return {"norm": _norm, "norm_grad": _norm_grad, "embed": _embed, "embed_grad": _embed_grad,
            "clip": _clip}[case["op"]](s, case)


def _norm(s, case):
    out, x = {}, s["x"]
    if case["residual"]:
        x = out["sum"] = (x.float() + s["residual"].float()).to(x.dtype)
    out["rstd"] = x.double().square().mean(1).add(EPS).rsqrt().float()
    v = x.float() * out["rstd"].unsqueeze(1) * s["w"].float()
    if case["values"]:
        out["y"] = v.to(x.dtype)
    if case["form"] in ("rows", "both"):
        out["rows"] = _quantized(v)
    if case["form"] in ("cols", "both"):
        out["cols"] = _quantized(v.t())
    return out


def _norm_grad(s, case):
    rstd = s["rstd"].unsqueeze(1)
    xh, dy = s["x"].float() * rstd, s["dy"].float()
    g = dy * s["w"].float()
    dx = (g - xh * (g * xh).mean(1, keepdim=True)) * rstd
    if case["past"]:
        dx = dx + s["past"].float()
    dw = (dy * xh).sum(0)
    return {"dx": dx.to(s["x"].dtype), "dw": s["dw"].add_(dw) if case["add"] else dw}


def _embed(s, case):
    t = s["tokens"].long()
    rows = s["table"][t.clamp(0, case["vocab"] - 1)].float() * case["scale"]
    live = (t >= 0) & (t < case["vocab"])
    return torch.where(live.unsqueeze(1), rows, torch.zeros_like(rows)).to(DTYPES[case["dtype"]])


def _embed_grad(s, case):
    t = s["tokens"].long()
    live = (t >= 0) & (t < case["vocab"])
    dy = torch.where(live.unsqueeze(1), s["dy"].float(), torch.zeros(1, device="cuda"))
    total = torch.zeros(case["vocab"], case["cols"], device="cuda")
    total.index_add_(0, t.clamp(0, case["vocab"] - 1), dy)
    return s["grad"].add_(total * case["scale"]) if case["add"] else total * case["scale"]


def _clip(s, case):
    squares = [g.float().square().sum(dtype=torch.float64) for g in s["gs"]]
    norm = torch.stack(squares).sum().sqrt().float()
    if case["ratio"] == 0.0:
        return {"norm": norm}
    some = (norm > s["max_norm"]) & torch.isfinite(norm)
    factor = torch.where(some, s["max_norm"] / norm.double(), 1.0).float()
    for g, o in zip(s["gs"], s["outs"] if case["out"] else s["gs"]):
        o.copy_(g.float() * factor)
    return {"norm": norm, "g": s["flat"]}


def _run_own(s, case, op):
    import decoupled_momentum_optimizer_gb300 as dm

    if op == "norm":
        form = None if case["form"] == "none" else case["form"]
        n = dm.rms_norm(s["x"], s["w"], eps=EPS, residual=s.get("residual"), values=case["values"], form=form, save=True)
        out = {"rstd": n.rstd}
        if case["residual"]:
            out["sum"] = n.total
        if case["values"]:
            out["y"] = n.out
        if form is not None:
            forms = n.quantized if form == "both" else (n.quantized,)
            for name, q in zip(("rows", "cols") if form == "both" else (form,), forms):
                out[name] = [q.codes, q.scales[:, :q.shape[0]]]
        return out
    if op == "norm_grad":
        dx, dw = dm.rms_norm_grad(s["dy"], s["x"], s["w"], s["rstd"], past=s.get("past"), dweight=s.get("dw"),
                                  add=case["add"])
        return {"dx": dx, "dw": dw}
    if op == "embed":
        return dm.embedding(s["tokens"], s["table"], scale=case["scale"], dtype=DTYPES[case["dtype"]])
    if op == "embed_grad":
        return dm.embedding_grad(s["tokens"], s["dy"], case["vocab"], scale=case["scale"], out=s.get("grad"),
                                 add=case["add"])
    if case["ratio"] == 0.0:
        return {"norm": dm.grad_norm(s["gs"])}
    return {"norm": dm.clip_grads(s["gs"], s["max_norm"], out=s.get("outs")), "g": s["flat"]}


# ---- the definitions in 64 bits ------------------------------------------------------------------

def _exact_codes(x):
    """(codes, scales) of x by rows, as float64 values."""
    rows, k = x.shape
    kb = -(-k // BLOCK)
    codes, scales = np.zeros((rows, kb * BLOCK)), np.ones((kb, rows))
    for b in range(kb):
        cols = slice(b * BLOCK, min(k, (b + 1) * BLOCK))
        amax = np.abs(x[:, cols]).max(1)
        e = np.zeros(rows)
        some = amax > 0
        e[some] = np.maximum(np.ceil(np.log2(amax[some] / 448.0)), -126)
        e[some & (amax > 448.0 * 2.0 ** e)] += 1  # the logarithm's rounding, next to a power of two
        e[some & (e > -126) & (amax <= 448.0 * 2.0 ** (e - 1))] -= 1
        scales[b] = 2.0 ** e
        v = x[:, cols] / scales[b][:, None]
        grain = 2.0 ** (np.maximum(np.frexp(v)[1] - 1, -6) - 3)
        codes[:, cols] = np.rint(v / grain) * grain
    return [torch.from_numpy(codes), torch.from_numpy(scales)]


def _host(t):
    return t.double().cpu().numpy()


def _exact_norm(s, case):
    x, w, out = _host(s["x"]), _host(s["w"]), {}
    if case["residual"]:
        out["sum"] = torch.from_numpy(x + _host(s["residual"]))
        x = _host(out["sum"].to(DTYPES[case["dtype"]]))  # the norm is defined on the stored sum
    rstd = 1.0 / np.sqrt(np.einsum("rc,rc->r", x, x) / case["cols"] + EPS)
    out["rstd"] = torch.from_numpy(rstd)
    if case["values"]:
        out["y"] = torch.from_numpy(x * rstd[:, None] * w)
    if case["form"] != "none":  # codes are defined on float32 products with the float32 rstd
        v = x.astype(np.float32) * rstd.astype(np.float32)[:, None] * w.astype(np.float32)
        v = v.astype(np.float64)
        if case["form"] != "cols":
            out["rows"] = _exact_codes(v)
        if case["form"] != "rows":
            out["cols"] = _exact_codes(np.ascontiguousarray(v.T))
    return out


def _exact_norm_grad(s, case):
    x, w, dy, rstd = s["x"].double(), s["w"].double(), s["dy"].double(), s["rstd"].double()
    dot = torch.einsum("rc,rc,c->r", dy, x, w)
    dx = torch.einsum("rc,c,r->rc", dy, w, rstd) - torch.einsum("rc,r->rc", x, dot * rstd ** 3 / case["cols"])
    if case["past"]:
        dx += s["past"].double()
    dw = torch.einsum("rc,rc,r->c", dy, x, rstd)
    return {"dx": dx, "dw": dw + s["dw"].double() if case["add"] else dw}


def _exact_embed(s, case):
    tokens, table = s["tokens"].cpu().numpy(), s["table"].cpu()
    live = np.flatnonzero((tokens >= 0) & (tokens < case["vocab"]))
    out = torch.zeros(len(tokens), case["cols"], dtype=torch.float64)
    out[torch.from_numpy(live)] = table[torch.from_numpy(tokens[live].astype(np.int64))].double() * case["scale"]
    return out


def _exact_embed_grad(s, case):
    tokens, dy = s["tokens"].cpu().numpy(), s["dy"].double()
    order = np.argsort(tokens, kind="stable")
    order = order[np.searchsorted(tokens[order], 0):np.searchsorted(tokens[order], case["vocab"])]
    out = torch.zeros(case["vocab"], case["cols"], dtype=torch.float64, device="cuda")
    if case["add"]:
        out += s["grad"].double()
    if len(order):
        rows, starts = np.unique(tokens[order], return_index=True)
        ends = np.append(starts[1:], len(order))
        sums = torch.empty(len(rows), case["cols"], dtype=torch.float64, device="cuda")
        running = dy[torch.from_numpy(order).cuda()].cumsum(0)
        sums.copy_(running[torch.from_numpy(ends - 1).cuda()])
        sums[1:] -= running[torch.from_numpy(starts[1:] - 1).cuda()]
        out[torch.from_numpy(rows.astype(np.int64)).cuda()] += sums * case["scale"]
    return out


def _exact_clip(s, case):
    total = math.fsum(torch.dot(g.double(), g.double()).item() for g in s["gs"])
    norm = math.sqrt(total)
    out = {"norm": torch.tensor(norm, dtype=torch.float64)}
    if case["ratio"] > 0.0:
        g = torch.zeros(s["flat"].shape, dtype=torch.float64, device="cuda") if case["out"] else s["flat"].double()
        for v, o in zip(s["gs"], s["outs"] if case["out"] else s["gs"]):
            at = o.storage_offset()
            g[at:at + v.numel()] = v.double() * min(1.0, s["max_norm"] / norm)
        out["g"] = g
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "embed": _exact_embed, "embed_grad": _exact_embed_grad,
            "clip": _exact_clip}[case["op"]](s, case)
