"""Training operators beside the shard step: dropout, 8-bit quantization and its products.

Bindings of ``demo_dropout``, ``demo_fp8_quantize``, ``demo_fp8_matmul`` and ``demo_fp8_linear``
(``include/demo.h``), in the package's manner: tensors are checked, results are allocated through
torch unless an ``out`` is given, the call runs on torch's current stream (or on ``stream``, as if it
were the current one) and raises :class:`DemoError` on a negative status.

The calls record nothing for autograd.  A tensor that requires a gradient is refused while gradients are
recorded (a result without history would end the branch's training without a word): call them from a
``torch.autograd.Function``, whose backward is the call that each docstring names, or under
``torch.no_grad()``.
"""

import functools

import torch

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
FP8_FORMATS = {"e4m3": (0, torch.float8_e4m3fn), "e5m2": (1, torch.float8_e5m2)}
_FMT_OF = {dt: code for code, dt in FP8_FORMATS.values()}
BLOCK = 128


class _Library:
    """The library's entry points, bound on first use (these calls are made per layer and step: the
    binding costs as much as a small kernel, so it looks nothing up twice)."""

    def __getattr__(self, name):
        import decoupled_momentum_optimizer_gb300 as dm

        setattr(self, name, getattr(dm, name[3:]) if name.startswith("dm_") else getattr(dm.lib(), name))
        return getattr(self, name)


_lib = _Library()
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _run(name, args, index):
    """Entry point ``name`` on ``args`` and device ``index``'s current stream, with the device current
    and initialised; raises on a negative status."""
    if index in _lib.dm__inited and _current_device() == index:
        raw = _raw_stream(index) if _raw_stream is not None else _lib.dm__stream(None, index)
        status = getattr(_lib, name)(*args, raw)
    else:
        with _lib.dm__OnDevice(torch.device("cuda", index)):
            status = getattr(_lib, name)(*args, _lib.dm__stream(None, index))
    if status:
        _lib.dm__check(status, name)


def _on_stream(stream, device, f, *args, **kw):
    """``f`` with ``stream`` current, so that what it allocates belongs to the stream it is used on."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream, device=device)
    elif stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the call's tensors on {device}")
    with torch.cuda.stream(stream):
        return f(*args, **kw)


def _matrix(t, name, like=None, shape=None):
    """(pointer, row stride, rows, columns) of a tensor seen as rows of its last dimension."""
    try:
        ptr, size, dt = t.data_ptr(), t.shape, t.dtype
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (there is no CPU path)")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, and this call records none: detach it, or call under "
                         "torch.no_grad() or from a torch.autograd.Function")
    if like is not None:
        if dt != like.dtype:
            raise TypeError(f"{name} has dtype {dt}, expected {like.dtype}")
        if t.get_device() != like.get_device():
            raise ValueError(f"{name} is on {t.device}, the call's other tensors on {like.device}")
        shape = like.shape
    elif dt not in _DTYPES:
        raise TypeError(f"{name} has dtype {dt}, expected float32, bfloat16 or float16")
    if shape is not None and size != shape:
        raise ValueError(f"{name} has shape {tuple(size)}, expected {tuple(shape)}")
    if len(size) == 2:
        rows, cols = size
        ld, inner = t.stride()
        if inner != 1 and cols > 1 and rows > 0:
            raise ValueError(f"{name}'s last dimension must be contiguous")
        return ptr, ld, rows, cols
    if not size:
        raise ValueError(f"{name} must have at least one dimension")
    cols = size[-1]
    rows = t.numel() // cols if cols else 0
    if cols > 1 and rows > 0 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    ld = cols
    if rows > 1 and not t.is_contiguous():  # leading dimensions that make one sequence of rows
        lead = [(n, s) for n, s in zip(size[:-1], t.stride()[:-1]) if n != 1]
        for (_, s), (n2, s2) in zip(lead, lead[1:]):
            if s != n2 * s2:
                raise ValueError(f"{name}'s leading dimensions must have one stride between rows")
        ld = lead[-1][1]
    return ptr, ld, rows, cols


def dropout(x, p, *, seed, step, site=0, residual=None, out=None, stream=None):
    """``residual + keep * x / (1 - p)`` (demo_dropout), the mask hashed from (seed, step, site,
    position) and never stored; rows are the last dimension.

    The gradient of ``x`` is ``dropout(dy, p, seed=..., step=..., site=...)`` with the same
    arguments; the residual's is ``dy``.  ``out`` may be ``x`` or ``residual`` themselves.
    """
    if stream is not None:
        return _on_stream(stream, x.device, dropout, x, p, seed=seed, step=step, site=site, residual=residual, out=out)
    xp, ldx, rows, cols = _matrix(x, "x")
    rp, ldr = _matrix(residual, "residual", x)[:2] if residual is not None else (None, 0)
    if out is None:
        out = torch.empty_like(x) if x.is_contiguous() else torch.empty(x.shape, dtype=x.dtype, device=x.device)
        op, ldo = out.data_ptr(), cols
    else:
        op, ldo = _matrix(out, "out", x)[:2]
    _run("demo_dropout", (xp, ldx, rp, ldr, op, ldo, _DTYPES[x.dtype], rows, cols, p, seed, step, site),
         x.get_device())
    return out


def _empty(rows, cols, dtype, device):
    """torch.empty, by the form of it that parses its arguments fastest."""
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


class Fp8Matrix:
    """A [rows, k] matrix in 8-bit floating point, a scale for each block of 128 along a row.

    ``codes``  float8 [rows, ceil(k / 128) * 128], zero past k
    ``scales`` float32 [ceil(k / 128), rows rounded up to 4]: element (r, c) is
               ``codes[r, c] * scales[c // 128, r]``.  Every scale is a power of two from 2^-126 to 2^127,
               as :func:`fp8_quantize` writes them (0 only where its block's codes are 0); the products
               make NaN of the results that any other scale takes part in.  ``check=True`` refuses
               such scales here (it waits for the device).
    ``tiles``  whether the scales are equal within each 128 rows as well
    """

    __slots__ = ("codes", "scales", "shape", "tiles")

    def __init__(self, codes, scales, k, *, tiles=False, check=False):
        if codes.dtype not in _FMT_OF or codes.dim() != 2:
            raise TypeError("codes must be a 2-D float8_e4m3fn or float8_e5m2 tensor")
        rows, width = codes.shape
        blocks = (k + BLOCK - 1) // BLOCK
        if width != blocks * BLOCK:
            raise ValueError(f"codes have {width} columns, expected {blocks * BLOCK} for k = {k}")
        if scales.dtype != torch.float32 or scales.shape != (blocks, (rows + 3) // 4 * 4):
            raise ValueError(f"scales must be float32 [{blocks}, {(rows + 3) // 4 * 4}]")
        if not codes.is_contiguous() or not scales.is_contiguous():
            raise ValueError("codes and scales must be contiguous")
        if not codes.is_cuda or scales.get_device() != codes.get_device():
            raise ValueError("codes and scales must be on one CUDA device (there is no CPU path)")
        if check:
            bits = scales[:, :rows].view(torch.int32)
            if not bool((((bits & -0x7f800001) == 0) & (bits != 0x7f800000)).all()):
                raise ValueError("scales must be powers of two from 2^-126 to 2^127 (or 0)")
        self.codes, self.scales, self.shape, self.tiles = codes, scales, (rows, k), tiles

    @classmethod
    def empty(cls, rows, k, fmt="e4m3", *, tiles=False, device="cuda"):
        """Uninitialised buffers of the right sizes, for fp8_quantize's ``out``."""
        q = cls.__new__(cls)
        blocks = (k + BLOCK - 1) // BLOCK
        q.codes = _empty(rows, blocks * BLOCK, FP8_FORMATS[fmt][1], device)
        q.scales = _empty(blocks, (rows + 3) // 4 * 4, torch.float32, device)
        q.shape, q.tiles = (rows, k), tiles
        return q

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
    if stream is not None:
        return _on_stream(stream, x.device, fp8_quantize, x, fmt=fmt, form=form, scales=scales, relu=relu, gate=gate, p=p,
                          seed=seed, step=step, site=site, out=out)
    if fmt not in FP8_FORMATS:
        raise ValueError(f"fmt is {fmt!r}, expected one of {tuple(FP8_FORMATS)}")
    if scales != "rows" and scales != "tiles":
        raise ValueError(f"scales is {scales!r}, expected rows or tiles")
    tiles = scales == "tiles"
    xp, ldx, rows, cols = _matrix(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x has {x.dim()} dimensions, expected 2")
    gp, ldg = _matrix(gate, "gate", x)[:2] if gate is not None else (None, 0)
    by_rows = by_cols = None
    if form == "both":
        by_rows, by_cols = out if out is not None else (None, None)
    elif form == "rows":
        by_rows = out
    elif form == "cols":
        by_cols = out
    else:
        raise ValueError(f"form is {form!r}, expected rows, cols or both")
    cr = sr = cc = sc = None
    if form != "cols":
        by_rows = _form(by_rows, rows, cols, fmt, tiles, x)
        cr, sr = by_rows.codes.data_ptr(), by_rows.scales.data_ptr()
    if form != "rows":
        by_cols = _form(by_cols, cols, rows, fmt, tiles, x)
        cc, sc = by_cols.codes.data_ptr(), by_cols.scales.data_ptr()
    _run("demo_fp8_quantize", (xp, ldx, _DTYPES[x.dtype], rows, cols, bool(relu), gp, ldg, p, seed, step, site,
                               FP8_FORMATS[fmt][0], tiles, cr, sr, cc, sc), x.get_device())
    return (by_rows, by_cols) if form == "both" else by_rows if by_cols is None else by_cols


def _form(q, rows, k, fmt, tiles, x):
    """A new Fp8Matrix [rows, k] beside x, or the given one if it is one."""
    if q is None:
        return Fp8Matrix.empty(rows, k, fmt, tiles=tiles, device=x.device)
    if q.shape != (rows, k) or q.codes.dtype != FP8_FORMATS[fmt][1] or q.tiles != tiles or \
            q.codes.get_device() != x.get_device():
        raise ValueError(f"out must be a {fmt} Fp8Matrix of shape {(rows, k)} with "
                         f"{'tiles' if tiles else 'rows'} scales on {x.device}")
    return q


def _out(out, shape, dtype, beside):
    """(out or a new tensor, pointer, row stride, dtype's code)."""
    if out is None:
        out = torch.empty(*shape, dtype=dtype, device=beside.device)
        return out, out.data_ptr(), shape[-1], _DTYPES[dtype]
    if dtype is not None and out.dtype != dtype:
        raise TypeError(f"out has dtype {out.dtype}, expected {dtype}")
    if out.get_device() != beside.get_device():
        raise ValueError(f"out is on {out.device}, the call's other tensors on {beside.device}")
    ptr, ld = _matrix(out, "out", None, shape)[:2]
    return out, ptr, ld, _DTYPES[out.dtype]


def _result_dtype(out, dtype, default):
    dtype = dtype if dtype is not None or out is not None else default
    if dtype is not None and dtype not in _DTYPES:
        raise TypeError(f"dtype is {dtype}, expected float32, bfloat16 or float16")
    return dtype


def fp8_matmul(a, b, *, out=None, dtype=None, add=False, stream=None):
    """``a b^T`` of two Fp8Matrix ([m, k] and [n, k]) into ``out`` or a new tensor of ``dtype``
    (bfloat16 by default), or added to the float32 ``out`` (demo_fp8_matmul).

    With ``dy`` the result's gradient, that of ``a`` is ``dy b`` and that of ``b`` is ``dy^T a``: products of
    ``dy`` quantized by rows, or by columns, with ``b``, or ``a``, quantized by columns.
    """
    if stream is not None:
        return _on_stream(stream, a.codes.device, fp8_matmul, a, b, out=out, dtype=dtype, add=add)
    (m, k), (n, kb) = a.shape, b.shape
    if k != kb:
        raise ValueError(f"a has k = {k}, b has k = {kb}")
    ac, bc = a.codes, b.codes
    index = ac.get_device()
    if bc.get_device() != index:
        raise ValueError(f"a is on {ac.device}, b on {bc.device}")
    if add and out is None:
        raise ValueError("add needs an out to add to")
    out, op, ldo, dt = _out(out, (m, n), _result_dtype(out, dtype, torch.bfloat16), ac)
    _run("demo_fp8_matmul", (ac.data_ptr(), a.scales.data_ptr(), _FMT_OF[ac.dtype], bc.data_ptr(),
                             b.scales.data_ptr(), _FMT_OF[bc.dtype], m, n, k, op, ldo, dt, bool(add)), index)
    return out


@functools.lru_cache(maxsize=1024)
def _linear_workspace(m, n, k):
    return _lib.demo_fp8_linear_workspace(m, n, k)


def fp8_linear(x, w, *, out=None, dtype=None, workspace=None, stream=None):
    """``x w^T`` for ``x`` [..., k] in 16 or 32 bits and an Fp8Matrix ``w`` [n, k] (demo_fp8_linear):
    ``x`` is quantized by rows to e4m3 within the call.  The result has x's dtype unless ``dtype``
    or ``out`` says otherwise; ``workspace`` (uint8, only used beyond a few rows) is allocated
    through torch where it is not given.  The gradients are those of :func:`fp8_matmul`.
    """
    if stream is not None:
        return _on_stream(stream, x.device, fp8_linear, x, w, out=out, dtype=dtype, workspace=workspace)
    xp, ldx, m, k = _matrix(x, "x")
    n, kw = w.shape
    if k != kw:
        raise ValueError(f"x has k = {k}, w has k = {kw}")
    wc, index = w.codes, x.get_device()
    if wc.get_device() != index:
        raise ValueError(f"w is on {wc.device}, x on {x.device}")
    lead = x.shape[:-1]
    if k == 0:
        m = lead.numel()
    out, op, ldo, odt = _out(out, (*lead, n), _result_dtype(out, dtype, x.dtype), x)
    need = _linear_workspace(m, n, k)
    wp = None
    if need:
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        elif workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.get_device() != index:
            raise ValueError(f"workspace must be a contiguous uint8 tensor on {x.device}")
        wp, need = workspace.data_ptr(), workspace.numel()
    _run("demo_fp8_linear", (xp, ldx, _DTYPES[x.dtype], wc.data_ptr(), w.scales.data_ptr(), _FMT_OF[wc.dtype], m, n, k,
                             op, ldo, odt, wp, need), index)
    return out
