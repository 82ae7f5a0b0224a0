"""Training operators beside the shard step: dropout, 8-bit quantization and its products.

Bindings of ``demo_dropout``, ``demo_fp8_quantize``, ``demo_fp8_matmul`` and ``demo_fp8_linear``
(``include/demo.h``), in the package's manner: tensors are checked, results are allocated through
torch unless an ``out`` is given, the call runs on torch's current stream (or ``stream``) and raises
:class:`DemoError` on a negative status.
"""

import ctypes

import torch

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
FP8_FORMATS = {"e4m3": (0, torch.float8_e4m3fn), "e5m2": (1, torch.float8_e5m2)}
_FMT_OF = {dt: code for code, dt in FP8_FORMATS.values()}
BLOCK = 128


def _pkg():
    import decoupled_momentum_optimizer_gb300 as dm

    return dm


def _dtype(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (there is no CPU path)")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} has dtype {t.dtype}, expected float32, bfloat16 or float16")
    return _DTYPES[t.dtype]


def _matrix(t, name, like=None, shape=None):
    """(pointer, row stride, rows, columns) of a tensor seen as rows of its last dimension."""
    dt = _dtype(t, name)
    if like is not None:
        if t.dtype != like.dtype:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {like.dtype}")
        if t.device != like.device:
            raise ValueError(f"{name} is on {t.device}, the call's other tensors on {like.device}")
        shape = like.shape
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dim() == 0:
        raise ValueError(f"{name} must have at least one dimension")
    cols = t.shape[-1]
    rows = t.numel() // cols if cols else 0
    if cols > 1 and rows > 0 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    ld = cols
    if rows > 1:
        if t.dim() == 2:
            ld = t.stride(0)
        elif not t.is_contiguous():  # leading dimensions that make one sequence of rows
            lead = [(n, s) for n, s in zip(t.shape[:-1], t.stride()[:-1]) if n != 1]
            for (_, s), (n2, s2) in zip(lead, lead[1:]):
                if s != n2 * s2:
                    raise ValueError(f"{name}'s leading dimensions must have one stride between rows")
            ld = lead[-1][1]
    return t.data_ptr(), ld, rows, cols, dt


def dropout(x, p, *, seed, step, site=0, residual=None, out=None, stream=None):
    """``residual + keep * x / (1 - p)`` (demo_dropout), the mask hashed from (seed, step, site,
    position) and never stored; rows are the last dimension.

    The gradient of ``x`` is ``dropout(dy, p, seed=..., step=..., site=...)`` with the same
    arguments; the residual's is ``dy``.  ``out`` may be ``x`` or ``residual`` themselves.
    """
    dm = _pkg()
    xp, ldx, rows, cols, dt = _matrix(x, "x")
    with dm._OnDevice(x.device) as d:
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        op, ldo = _matrix(out, "out", like=x)[:2]
        rp, ldr = _matrix(residual, "residual", like=x)[:2] if residual is not None else (None, 0)
        dm._check(dm.lib().demo_dropout(xp, ldx, rp, ldr, op, ldo, dt, rows, cols, p, seed, step, site,
                                        dm._stream(stream, d.index)), "demo_dropout")
    return out


class Fp8Matrix:
    """A [rows, k] matrix in 8-bit floating point, a scale for each block of 128 along a row.

    ``codes``  float8 [rows, ceil(k / 128) * 128], zero past k
    ``scales`` float32 [ceil(k / 128), rows rounded up to 4]: element (r, c) is
               ``codes[r, c] * scales[c // 128, r]``
    ``tiles``  whether the scales are equal within each 128 rows as well
    """

    __slots__ = ("codes", "scales", "shape", "tiles")

    def __init__(self, codes, scales, k, *, tiles=False):
        if codes.dim() != 2 or codes.dtype not in _FMT_OF:
            raise TypeError("codes must be a 2-D float8_e4m3fn or float8_e5m2 tensor")
        rows, blocks = codes.shape[0], (k + BLOCK - 1) // BLOCK
        if codes.shape[1] != blocks * BLOCK:
            raise ValueError(f"codes have {codes.shape[1]} columns, expected {blocks * BLOCK} for k = {k}")
        if scales.dtype != torch.float32 or tuple(scales.shape) != (blocks, (rows + 3) // 4 * 4):
            raise ValueError(f"scales must be float32 [{blocks}, {(rows + 3) // 4 * 4}]")
        if not codes.is_contiguous() or not scales.is_contiguous():
            raise ValueError("codes and scales must be contiguous")
        if not codes.is_cuda or scales.device != codes.device:
            raise ValueError("codes and scales must be on one CUDA device (there is no CPU path)")
        self.codes, self.scales, self.shape, self.tiles = codes, scales, (rows, k), bool(tiles)

    @classmethod
    def empty(cls, rows, k, fmt="e4m3", *, tiles=False, device="cuda"):
        """Uninitialised buffers of the right sizes, for fp8_quantize's ``out``."""
        kp = (k + BLOCK - 1) // BLOCK * BLOCK
        codes = torch.empty(rows, kp, dtype=FP8_FORMATS[fmt][1], device=device)
        return cls(codes, torch.empty(kp // BLOCK, (rows + 3) // 4 * 4, device=device), k, tiles=tiles)

    def dequantize(self):
        """The float32 values (torch operations: for tests and inspection)."""
        rows, k = self.shape
        v = self.codes.float().view(rows, -1, BLOCK) * self.scales[:, :rows].t().unsqueeze(2)
        return v.reshape(rows, -1)[:, :k]


def fp8_quantize(x, *, fmt="e4m3", form="rows", scales="rows", relu=False, gate=None, p=0.0, seed=0, step=0, site=0,
                 out=None, stream=None):
    """Quantize a 2-D tensor to an :class:`Fp8Matrix` (demo_fp8_quantize).

    ``form``   "rows" (x itself), "cols" (its transpose) or "both" (a pair, from one read of x)
    ``scales`` "rows": one for 128 elements along the form's rows; "tiles": one for 128 x 128
    ``relu``, ``p`` (with ``seed``, ``step``, ``site`` as for :func:`dropout`) and ``gate`` are
    applied on the way in, in this order; ``gate`` zeroes the elements where it is not positive.
    ``out``    the Fp8Matrix, or the pair, to write into
    """
    dm = _pkg()
    if form not in ("rows", "cols", "both"):
        raise ValueError(f"form is {form!r}, expected rows, cols or both")
    if scales not in ("rows", "tiles"):
        raise ValueError(f"scales is {scales!r}, expected rows or tiles")
    if fmt not in FP8_FORMATS:
        raise ValueError(f"fmt is {fmt!r}, expected one of {tuple(FP8_FORMATS)}")
    xp, ldx, _, _, dt = _matrix(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x has {x.dim()} dimensions, expected 2")
    rows, cols = x.shape
    tiles = scales == "tiles"
    with dm._OnDevice(x.device) as d:
        gp, ldg = _matrix(gate, "gate", like=x)[:2] if gate is not None else (None, 0)
        shapes = [s for f, s in (("rows", (rows, cols)), ("cols", (cols, rows))) if form in (f, "both")]
        if out is None:
            qs = [Fp8Matrix.empty(*s, fmt, tiles=tiles, device=x.device) for s in shapes]
        else:
            qs = list(out) if form == "both" else [out]
            for q, s in zip(qs, shapes):
                if q.shape != s or q.codes.dtype != FP8_FORMATS[fmt][1] or q.tiles != tiles or \
                        q.codes.device != x.device:
                    raise ValueError(f"out must be a {fmt} Fp8Matrix of shape {s} with {scales} scales on {x.device}")
            if len(qs) != len(shapes):
                raise ValueError("out must be a pair for form='both'")
        ptrs = [None] * 4
        for i, q in enumerate(qs):
            at = 2 if form == "cols" else 2 * i
            ptrs[at], ptrs[at + 1] = q.codes.data_ptr(), q.scales.data_ptr()
        dm._check(dm.lib().demo_fp8_quantize(xp, ldx, dt, rows, cols, int(bool(relu)), gp, ldg, p, seed, step, site,
                                             FP8_FORMATS[fmt][0], int(tiles), *ptrs, dm._stream(stream, d.index)),
                  "demo_fp8_quantize")
    return tuple(qs) if form == "both" else qs[0]


def _out(out, shape, dtype, device):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if dtype is not None and out.dtype != dtype:
        raise TypeError(f"out has dtype {out.dtype}, expected {dtype}")
    if out.device != device:
        raise ValueError(f"out is on {out.device}, the call's other tensors on {device}")
    return out


def fp8_matmul(a, b, *, out=None, dtype=None, add=False, stream=None):
    """``a b^T`` of two Fp8Matrix ([m, k] and [n, k]) into ``out`` or a new tensor of ``dtype``
    (bfloat16 by default), or added to the float32 ``out`` (demo_fp8_matmul)."""
    dm = _pkg()
    if a.shape[1] != b.shape[1]:
        raise ValueError(f"a has k = {a.shape[1]}, b has k = {b.shape[1]}")
    if a.codes.device != b.codes.device:
        raise ValueError(f"a is on {a.codes.device}, b on {b.codes.device}")
    if add and out is None:
        raise ValueError("add needs an out to add to")
    (m, k), n = a.shape, b.shape[0]
    with dm._OnDevice(a.codes.device) as d:
        out = _out(out, (m, n), dtype or (None if out is not None else torch.bfloat16), a.codes.device)
        op, ldo, _, _, dt = _matrix(out, "out", shape=(m, n))
        dm._check(dm.lib().demo_fp8_matmul(a.codes.data_ptr(), a.scales.data_ptr(), _FMT_OF[a.codes.dtype],
                                           b.codes.data_ptr(), b.scales.data_ptr(), _FMT_OF[b.codes.dtype],
                                           m, n, k, op, ldo, dt, int(bool(add)), dm._stream(stream, d.index)), "demo_fp8_matmul")
    return out


def fp8_linear(x, w, *, out=None, dtype=None, workspace=None, stream=None):
    """``x w^T`` for ``x`` [..., k] in 16 or 32 bits and an Fp8Matrix ``w`` [n, k] (demo_fp8_linear):
    ``x`` is quantized by rows to e4m3 within the call.  The result has x's dtype unless ``dtype``
    or ``out`` says otherwise; ``workspace`` (uint8, only used beyond a few rows) is allocated
    through torch where it is not given.
    """
    dm = _pkg()
    xp, ldx, m, k, dt = _matrix(x, "x")
    n = w.shape[0]
    if k != w.shape[1]:
        raise ValueError(f"x has k = {k}, w has k = {w.shape[1]}")
    if w.codes.device != x.device:
        raise ValueError(f"w is on {w.codes.device}, x on {x.device}")
    if k == 0:
        m = x.shape[:-1].numel()
    with dm._OnDevice(x.device) as d:
        shape = (*x.shape[:-1], n)
        out = _out(out, shape, dtype or (None if out is not None else x.dtype), x.device)
        op, ldo, _, _, odt = _matrix(out, "out", shape=shape)
        need = dm.lib().demo_fp8_linear_workspace(m, n, k)
        if need and workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        wp, wn = (workspace.data_ptr(), workspace.numel()) if need else (None, 0)
        if need and (workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.device != x.device):
            raise ValueError(f"workspace must be a contiguous uint8 tensor on {x.device}")
        dm._check(dm.lib().demo_fp8_linear(xp, ldx, dt, w.codes.data_ptr(), w.scales.data_ptr(), _FMT_OF[w.codes.dtype],
                                           m, n, k, op, ldo, odt, wp, wn,
                                           dm._stream(stream, d.index)), "demo_fp8_linear")
    return out


_c_i64, _c_u64, _c_vp, _c_int, _c_f64 = ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p, ctypes.c_int, ctypes.c_double
SIGS = {
    "demo_dropout": (_c_int, [_c_vp, _c_i64, _c_vp, _c_i64, _c_vp, _c_i64, _c_int, _c_i64, _c_i64, _c_f64, _c_u64,
                              _c_u64, _c_u64, _c_vp]),
    "demo_fp8_bytes": (ctypes.c_size_t, [_c_i64, _c_i64, ctypes.POINTER(ctypes.c_size_t)]),
    "demo_fp8_quantize": (_c_int, [_c_vp, _c_i64, _c_int, _c_i64, _c_i64, _c_int, _c_vp, _c_i64, _c_f64, _c_u64,
                                   _c_u64, _c_u64, _c_int, _c_int, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp]),
    "demo_fp8_matmul": (_c_int, [_c_vp, _c_vp, _c_int, _c_vp, _c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_i64,
                                 _c_int, _c_int, _c_vp]),
    "demo_fp8_linear_workspace": (ctypes.c_size_t, [_c_i64, _c_i64, _c_i64]),
    "demo_fp8_linear": (_c_int, [_c_vp, _c_i64, _c_int, _c_vp, _c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_i64,
                                 _c_int, _c_vp, ctypes.c_size_t, _c_vp]),
}
