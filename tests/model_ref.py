"""Definitions in 64 bits (numpy) of the operators between the products and the step, from include/demo.h alone."""

import numpy as np
import torch

import train_ref as ref

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # half a step, relative
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}  # the smallest step


def f64(t):
    return t.double().cpu().numpy()


def draw(rows, cols, dtype="f32", seed=0, std=1.0, pad=0, offset=0, device="cuda"):
    """A [rows, cols] view whose rows are `pad` longer and start `offset` elements into the buffer."""
    gen = torch.Generator().manual_seed(seed)
    w = cols + pad
    x = torch.randn(rows * w + offset, generator=gen) * std
    x = x * torch.exp(0.5 * torch.randn(rows * w + offset, generator=gen))
    return x.to(DT[dtype]).to(device)[offset:].view(rows, w)[:, :cols]


def guarded(rows, cols, dtype, pad, offset):
    """As draw's views, over a buffer of a value that nothing computes; and a check that it is intact."""
    buf = torch.full(((rows * (cols + pad)) + offset + 8,), 12345.0, dtype=DT[dtype], device="cuda")
    view = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    inside = torch.zeros_like(buf, dtype=torch.bool)
    inside.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(True)
    return view, lambda: bool((buf[~inside] == 12345.0).all())


def rounded(v, dtype):
    """float32 or float64 values to the nearest of the type, as float64."""
    return torch.from_numpy(np.ascontiguousarray(v)).to(DT[dtype]).double().numpy()


# ---- norm ----------------------------------------------------------------------------------------

def norm_rstd(s, eps):
    """1 / sqrt(mean(s^2) + eps) of each row, in 64 bits."""
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        return 1.0 / np.sqrt(np.square(s).mean(1) + eps)


def norm_values(s, rstd32, w):
    """(s r) w in two float32 products, from the float32 factors."""
    with np.errstate(invalid="ignore", over="ignore"):
        return s.astype(np.float32) * rstd32.astype(np.float32)[:, None] * w.astype(np.float32)


def norm_grad(dy, s, w, rstd, past=None):
    """(dx, dw) and the sums of magnitudes (of dx's row sum, of dw) that bound float32's roundings."""
    xh = s * rstd[:, None]
    g = dy * w
    c = (g * xh).mean(1, keepdims=True)
    dx = rstd[:, None] * (g - xh * c)
    if past is not None:
        dx = dx + past
    return dx, (dy * xh).sum(0), np.abs(g * xh).sum(1, keepdims=True), np.abs(dy * xh).sum(0)


def norm_grad_tolerance(dy, s, w, rstd, past, dtype, rows_added):
    """Elementwise bounds of dx and dw.

    The row's sum: each of its terms is a product of three rounded factors and joins a sum of at most 32
    terms in a lane, then ten joins of lanes and warps: 3 + 32 + 10 roundings of the sum of magnitudes; two
    more for c.  dx then rounds xh, dy w, their difference, the product with rstd and the addition, and is
    rounded to its type.  dw: two roundings a term and one for each addition to a sum of `rows_added`.
    """
    dx, dw, row_sum, col_sum = norm_grad(dy, s, w, rstd, past)
    u = 2.0 ** -24
    xh, g, r = np.abs(s * rstd[:, None]), np.abs(dy * w), np.abs(rstd[:, None])
    c = row_sum / s.shape[1]
    tol = r * (xh * c * 47 * u + 4 * u * (g + xh * c)) + u * np.abs(dx) + u * (0 if past is None else np.abs(past))
    tol = tol * 1.01 + np.abs(dx) * HALF[dtype] + TINY[dtype]
    return tol, (rows_added + 2) * u * col_sum + 2.0 ** -140
