"""Training operators beside the shard step: embedding, norms, dropout, 8-bit quantization and its products,
and the clipping of what they leave.

Bindings of ``demo_dropout``, ``demo_fp8_quantize``, ``demo_fp8_matmul``, ``demo_fp8_linear``, ``demo_rms_norm``,
``demo_rms_norm_grad``, ``demo_embedding``, ``demo_embedding_grad``, ``demo_grad_norm`` and ``demo_clip_grads``
(``include/demo.h``), in the package's manner: tensors are checked, results are allocated through
torch unless an ``out`` is given, the call runs on torch's current stream (or on ``stream``, as if it
were the current one) and raises :class:`DemoError` on a negative status.

The calls record nothing for autograd.  A tensor that requires a gradient is refused while gradients are
recorded (a result without history would end the branch's training without a word), and so is one with a
forward-mode tangent: call them from a ``torch.autograd.Function``, whose backward is the call that each docstring
names, or, without a tangent, under ``torch.no_grad()``.  What a call writes of the tensors that it is given counts as
modified in place, as with torch's own ``out=`` (slices of a buffer share the count).
"""

import collections
import ctypes
import functools
import warnings

import torch
import torch.autograd.forward_ad as _forward_ad

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


@functools.lru_cache(maxsize=1)
def _extension():
    """The extension module (csrc/bind_ops.cpp), or None, with one warning, where there is none for this torch."""
    import decoupled_momentum_optimizer_gb300 as dm
    from decoupled_momentum_optimizer_gb300 import build

    dm.lib()
    try:
        from decoupled_momentum_optimizer_gb300 import _bind_ops
    except ImportError as e:
        why = str(e)
    else:  # it reads tensors as the torch that it was built against lays them out
        built, here = getattr(_bind_ops, "torch", "another torch"), build.torch_tag(torch)
        if built == here:
            return _bind_ops
        why = f"built against torch {built}, not {here}"
    warnings.warn(f"no extension module for this torch ({why}): norm, embedding and clipping calls go through ctypes, which "
                  "costs small ones several times as much.  Build it with python -m decoupled_momentum_optimizer_gb300.build",
                  RuntimeWarning, stacklevel=4)
    return None


def _declined(*args):
    return NotImplemented


class _Bindings:
    """The extension module's functions, bound on first use.  They take the plain calls, several times faster than
    ctypes does, and answer NotImplemented to all others, which the Python code below each of their calls then
    takes or refuses; without the module that code takes every call."""

    def __getattr__(self, name):
        module = _extension()
        setattr(self, name, _declined if module is None else getattr(module, name))
        return getattr(self, name)


_bind = _Bindings()


def _refused(status, name):
    """Raises for the status that a call of the extension module came back with."""
    _lib.dm__check(status, name)


# What a call writes of the tensors that it is given counts as modified in place, so that autograd notices where it saved
# one of them before.
_wrote = torch.autograd.graph.increment_version


def _written(*given):
    for t in given:
        if t is not None:
            _wrote((t.codes, t.scales) if t.__class__ is Fp8Matrix or not isinstance(t, torch.Tensor) else t)


_FORM_CODES = {None: 0, "rows": 1, "cols": 2, "both": 3}
_FMT_CODES = {"e4m3": 0, "e5m2": 1}
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


def _unfollowed(t, name):
    """Refuses a tensor that autograd follows: backward, or forward while a level of tangents is open."""
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, and this call records none: detach it, or call under "
                         "torch.no_grad() or from a torch.autograd.Function")
    if _forward_ad._current_level >= 0 and torch._C._is_fwd_grad_enabled() and _forward_ad.unpack_dual(t).tangent is not None:
        raise ValueError(f"{name} has a forward-mode tangent, and this call computes none: detach it, or call from a "
                         "torch.autograd.Function")


def _matrix(t, name, like=None, shape=None):
    """(pointer, row stride, rows, columns) of a tensor seen as rows of its last dimension."""
    try:
        ptr, size, dt = t.data_ptr(), t.shape, t.dtype
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (there is no CPU path)")
    if t.requires_grad or _forward_ad._current_level >= 0:
        _unfollowed(t, name)
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
    given = out
    if out is None:
        out = torch.empty_like(x) if x.is_contiguous() else torch.empty(x.shape, dtype=x.dtype, device=x.device)
        op, ldo = out.data_ptr(), cols
    else:
        op, ldo = _matrix(out, "out", x)[:2]
    _run("demo_dropout", (xp, ldx, rp, ldr, op, ldo, _DTYPES[x.dtype], rows, cols, p, seed, step, site),
         x.get_device())
    if given is not None:
        _wrote(given)
    return out


def _empty(rows, cols, dtype, device):
    """torch.empty, by the form of it that parses its arguments fastest."""
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _made(codes, scales, rows, k):
    """An Fp8Matrix of buffers that are known to be right."""
    q = Fp8Matrix.__new__(Fp8Matrix)
    q.codes, q.scales, q.shape, q.tiles = codes, scales, (rows, k), False
    return q


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
    given = by_rows, by_cols
    if form != "cols":
        by_rows = _form(by_rows, rows, cols, fmt, tiles, x)
        cr, sr = by_rows.codes.data_ptr(), by_rows.scales.data_ptr()
    if form != "rows":
        by_cols = _form(by_cols, cols, rows, fmt, tiles, x)
        cc, sc = by_cols.codes.data_ptr(), by_cols.scales.data_ptr()
    _run("demo_fp8_quantize", (xp, ldx, _DTYPES[x.dtype], rows, cols, bool(relu), gp, ldg, p, seed, step, site,
                               FP8_FORMATS[fmt][0], tiles, cr, sr, cc, sc), x.get_device())
    if out is not None:
        _written(*given)
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
    given = out
    out, op, ldo, dt = _out(out, (m, n), _result_dtype(out, dtype, torch.bfloat16), ac)
    _run("demo_fp8_matmul", (ac.data_ptr(), a.scales.data_ptr(), _FMT_OF[ac.dtype], bc.data_ptr(),
                             b.scales.data_ptr(), _FMT_OF[bc.dtype], m, n, k, op, ldo, dt, bool(add)), index)
    if given is not None:
        _wrote(given)
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
    given = out
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
    if given is not None:
        _wrote(given)
    return out


Normed = collections.namedtuple("Normed", ("out", "quantized", "total", "rstd"))


def _flat_rows(t):
    """Rows of a tensor seen as rows of its last dimension (also where that has no elements)."""
    return t.shape[:-1].numel()


def _weight(weight, x, cols):
    """(pointer, dtype's code) of a norm's weight: [cols], contiguous, float32 or x's type."""
    if weight.dtype != torch.float32 and weight.dtype != x.dtype:
        raise TypeError(f"weight has dtype {weight.dtype}, expected float32 or {x.dtype}")
    if weight.get_device() != x.get_device():
        raise ValueError(f"weight is on {weight.device}, x on {x.device}")
    return _matrix(weight, "weight", None, (cols,))[0], _DTYPES[weight.dtype]


def _row_values(t, name, rows, beside):
    """Pointer of a contiguous float32 tensor with one element a row."""
    if t.dtype != torch.float32 or t.numel() != rows or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of {rows} elements")
    if t.get_device() != beside.get_device():
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on {beside.device}")
    if t.requires_grad or _forward_ad._current_level >= 0:
        _unfollowed(t, name)
    return t.data_ptr()


def _workspace(workspace, need, beside):
    """(tensor, pointer, bytes) of a call's workspace: the given one, or a new one where it needs any."""
    if not need:
        return None, None, 0
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=beside.device)
    elif workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.get_device() != beside.get_device():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {beside.device}")
    return workspace, workspace.data_ptr(), workspace.numel()


def rms_norm(x, weight, *, eps=1e-6, residual=None, values=True, form=None, fmt="e4m3", save=False, out=None, total=None,
             rstd=None, quantized=None, stream=None):
    """Root-mean-square norm of the last dimension with the residual's addition before it (demo_rms_norm):
    ``total = x + residual`` and ``out = total / sqrt(mean(total^2) + eps) * weight``.

    ``weight``  [cols], float32 (a slice of the flat shard) or x's type
    ``values``  whether ``out``, in x's type, is written
    ``form``    None, or "rows", "cols", "both": the result as an :class:`Fp8Matrix` (or the pair), of the
                values before their rounding to x's type, as :func:`fp8_quantize` makes them (2-D x)
    ``save``    whether the rows' factors ``rstd``, which :func:`rms_norm_grad` takes, are returned
    ``out``, ``total``, ``rstd``, ``quantized``   where the results go; new tensors otherwise.  ``total`` and
                ``out`` may be ``x`` or ``residual`` themselves (``out`` not with "cols" or "both")

    Returns ``Normed(out, quantized, total, rstd)``: ``total`` is ``x`` without a residual, what was not asked
    for is None.
    """
    if stream is None and quantized is None:
        r = _bind.rms_norm(x, weight, eps, residual, values, _FORM_CODES.get(form, -1), _FMT_CODES.get(fmt, -1), save, out, total,
                           rstd)
        if r.__class__ is tuple:
            if form is None:
                return Normed(r[0], None, r[1], r[2])
            out, total, rstd, codes, scales, codes_cols, scales_cols, rows, cols = r
            if form == "rows":
                q = _made(codes, scales, rows, cols)
            elif form == "cols":
                q = _made(codes_cols, scales_cols, cols, rows)
            else:
                q = _made(codes, scales, rows, cols), _made(codes_cols, scales_cols, cols, rows)
            return Normed(out, q, total, rstd)
        if r is not NotImplemented:
            _refused(r, "demo_rms_norm")
    if stream is not None:
        return _on_stream(stream, x.device, rms_norm, x, weight, eps=eps, residual=residual, values=values, form=form, fmt=fmt,
                          save=save, out=out, total=total, rstd=rstd, quantized=quantized)
    if fmt not in FP8_FORMATS:
        raise ValueError(f"fmt is {fmt!r}, expected one of {tuple(FP8_FORMATS)}")
    xp, ldx, rows, cols = _matrix(x, "x")
    wp, wdt = _weight(weight, x, cols)
    rp, ldr, tp, ldt = None, 0, None, 0
    given = [out, total, rstd]
    if residual is not None:
        rp, ldr = _matrix(residual, "residual", x)[:2]
        if total is None:
            total = torch.empty(x.shape, dtype=x.dtype, device=x.device)
            tp, ldt = total.data_ptr(), cols
        else:
            tp, ldt = _matrix(total, "total", x)[:2]
    elif total is not None:
        raise ValueError("total is for a residual's sum")
    op, ldo = None, 0
    if out is not None:
        op, ldo = _matrix(out, "out", x)[:2]
    elif values:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        op, ldo = out.data_ptr(), cols
    by_rows = by_cols = cr = sr = cc = sc = None
    if form is not None:
        if x.dim() != 2:
            raise ValueError(f"x has {x.dim()} dimensions, expected 2 for the 8-bit forms")
        if form == "both":
            by_rows, by_cols = quantized if quantized is not None else (None, None)
        elif form == "rows":
            by_rows = quantized
        elif form == "cols":
            by_cols = quantized
        else:
            raise ValueError(f"form is {form!r}, expected rows, cols or both")
        given += by_rows, by_cols
        if form != "cols":
            by_rows = _form(by_rows, rows, cols, fmt, False, x)
            cr, sr = by_rows.codes.data_ptr(), by_rows.scales.data_ptr()
        if form != "rows":
            by_cols = _form(by_cols, cols, rows, fmt, False, x)
            cc, sc = by_cols.codes.data_ptr(), by_cols.scales.data_ptr()
    elif quantized is not None:
        raise ValueError("quantized needs a form")
    factors = rstd
    if rstd is None and (save or by_cols is not None):
        factors = torch.empty(_flat_rows(x), dtype=torch.float32, device=x.device)
    sp = _row_values(factors, "rstd", _flat_rows(x), x) if factors is not None else None
    _run("demo_rms_norm", (xp, ldx, rp, ldr, _DTYPES[x.dtype], wp, wdt, rows, cols, eps, tp, ldt, op, ldo, sp,
                           FP8_FORMATS[fmt][0], cr, sr, cc, sc), x.get_device())
    _written(*given)
    return Normed(out, (by_rows, by_cols) if form == "both" else by_cols if by_rows is None else by_rows,
                  x if residual is None else total, factors if save or rstd is not None else None)


@functools.lru_cache(maxsize=1024)
def _norm_workspace(rows, cols):
    return _lib.demo_rms_norm_grad_workspace(rows, cols)


def rms_norm_grad(dy, total, weight, rstd, *, past=None, out=None, dweight=None, add=False, weight_grad=True,
                  workspace=None, stream=None):
    """The gradients of :func:`rms_norm` (demo_rms_norm_grad): ``(dx, dweight)``.

    ``dy`` is the result's gradient (for an 8-bit result, that of the values its codes stand for),
    ``total`` and ``rstd`` are what the forward call returned; ``past`` is the gradient that reaches ``total``
    by other ways, added to ``dx``.  ``dx`` is the gradient of both ``x`` and ``residual``; ``out`` receives it
    and may be ``dy``, ``total`` or ``past`` themselves.  ``dweight`` is float32 [cols], written or (``add``)
    added to; with ``weight_grad=False`` it is left out and None.
    """
    if stream is None and workspace is None:
        r = _bind.rms_norm_grad(dy, total, weight, rstd, past, out, dweight, add, weight_grad)
        if r.__class__ is tuple:
            return r
        if r is not NotImplemented:
            _refused(r, "demo_rms_norm_grad")
    if stream is not None:
        return _on_stream(stream, dy.device, rms_norm_grad, dy, total, weight, rstd, past=past, out=out, dweight=dweight,
                          add=add, weight_grad=weight_grad, workspace=workspace)
    dp, ldd, rows, cols = _matrix(dy, "dy")
    tp, ldt = _matrix(total, "total", dy)[:2]
    wp, wdt = _weight(weight, dy, cols)
    sp = _row_values(rstd, "rstd", _flat_rows(dy), dy)
    pp, ldp = _matrix(past, "past", dy)[:2] if past is not None else (None, 0)
    given = out, dweight
    if out is None:
        out = torch.empty(dy.shape, dtype=dy.dtype, device=dy.device)
        op, ldo = out.data_ptr(), cols
    else:
        op, ldo = _matrix(out, "out", dy)[:2]
    gp = work = wsp = None
    need = 0
    if weight_grad:
        if dweight is None:
            if add:
                raise ValueError("add needs a dweight to add to")
            dweight = torch.empty(cols, dtype=torch.float32, device=dy.device)
        gp = _row_values(dweight, "dweight", cols, dy)
        work, wsp, need = _workspace(workspace, _norm_workspace(rows, cols), dy)
    elif dweight is not None:
        raise ValueError("dweight is given, and weight_grad is False")
    _run("demo_rms_norm_grad", (dp, ldd, tp, ldt, _DTYPES[dy.dtype], wp, wdt, sp, rows, cols, pp, ldp, op, ldo, gp, bool(add),
                                wsp, need), dy.get_device())
    _written(*given)
    return out, dweight


def _tokens(t):
    """(pointer, bytes a token, rows, tokens a row, row stride) of an integer tensor of any shape."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("tokens must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("tokens must be on a CUDA device (there is no CPU path)")
    size = 8 if t.dtype == torch.int64 else 4 if t.dtype == torch.int32 else 0
    if not size:
        raise TypeError(f"tokens have dtype {t.dtype}, expected int32 or int64")
    n = t.numel()
    if t.is_contiguous() or n <= 1:
        return t.data_ptr(), size, 1, n, n
    # Dimensions that make one run of tokens are one; what is left is a run, or rows of runs.
    runs = []
    for length, stride in zip(t.shape, t.stride()):
        if length == 1:
            continue
        if runs and runs[-1][1] == length * stride:
            runs[-1] = (runs[-1][0] * length, stride)
        else:
            runs.append((length, stride))
    if len(runs) == 1:
        return t.data_ptr(), size, n, 1, runs[0][1]
    if len(runs) == 2 and runs[1][1] == 1:
        return t.data_ptr(), size, runs[0][0], runs[1][0], runs[0][1]
    raise ValueError("tokens must be rows of consecutive ones with one stride between rows")


def embedding(tokens, table, *, scale=1.0, dtype=None, out=None, stream=None):
    """``scale * table[tokens]`` (demo_embedding) as [*tokens.shape, cols]: rows of a [vocab, cols] table in
    ``dtype`` (the table's by default), zeros for tokens outside [0, vocab).

    The gradient of the table is :func:`embedding_grad`.
    """
    if stream is None:
        r = _bind.embedding(tokens, table, scale, dtype, out)
        if r.__class__ is int:
            _refused(r, "demo_embedding")
        if r is not NotImplemented:
            return r
    if stream is not None:
        return _on_stream(stream, table.device, embedding, tokens, table, scale=scale, dtype=dtype, out=out)
    kp, size, krows, kcols, ldk = _tokens(tokens)
    tp, ldt, vocab, cols = _matrix(table, "table")
    if table.dim() != 2:
        raise ValueError(f"table has {table.dim()} dimensions, expected 2")
    if tokens.get_device() != table.get_device():
        raise ValueError(f"tokens are on {tokens.device}, the table on {table.device}")
    given = out
    out, op, ldo, odt = _out(out, (*tokens.shape, cols), _result_dtype(out, dtype, table.dtype), table)
    _run("demo_embedding", (kp, size, krows, kcols, ldk, tp, ldt, _DTYPES[table.dtype], vocab, cols, scale, op, ldo, odt),
         table.get_device())
    _written(given)
    return out


@functools.lru_cache(maxsize=1024)
def _embedding_workspace(n, cols):
    return _lib.demo_embedding_grad_workspace(n, cols)


def embedding_grad(tokens, dy, vocab=None, *, scale=1.0, out=None, add=False, workspace=None, stream=None):
    """The gradient of :func:`embedding`'s table (demo_embedding_grad), float32 [vocab, cols]: ``scale`` times the
    sum of the rows of ``dy`` [*tokens.shape, cols] for each token, in an order that the tokens, their number and cols
    decide.

    ``out``   a float32 [vocab, cols] to write (a slice of the flat gradient, say); a new tensor otherwise.  With
              ``add`` the sums are added to it, and rows that no token names stay as they are.
    ``workspace``   uint8; allocated through torch where it is not given
    """
    if stream is None and workspace is None:
        r = _bind.embedding_grad(tokens, dy, vocab, scale, out, add)
        if r.__class__ is int:
            _refused(r, "demo_embedding_grad")
        if r is not NotImplemented:
            return r
    if stream is not None:
        return _on_stream(stream, dy.device, embedding_grad, tokens, dy, vocab, scale=scale, out=out, add=add,
                          workspace=workspace)
    kp, size, krows, kcols, ldk = _tokens(tokens)
    dp, ldd, n, cols = _matrix(dy, "dy")
    if dy.shape[:-1] != tokens.shape:
        raise ValueError(f"dy has shape {tuple(dy.shape)}, expected {(*tokens.shape, cols)}")
    if tokens.get_device() != dy.get_device():
        raise ValueError(f"tokens are on {tokens.device}, dy on {dy.device}")
    if out is None:
        if vocab is None or add:
            raise ValueError("add needs an out to add to" if add else "vocab or out is needed")
    elif out.dim() != 2 or (vocab is not None and vocab != out.shape[0]):
        raise ValueError(f"out has shape {tuple(out.shape)}, expected [{'vocab' if vocab is None else vocab}, {cols}]")
    else:
        vocab = out.shape[0]
    given = out
    out, gp, ldg, _ = _out(out, (vocab, cols), torch.float32, dy)
    workspace, wsp, need = _workspace(workspace, _embedding_workspace(n, cols), dy)
    _run("demo_embedding_grad", (kp, size, krows, kcols, ldk, dp, ldd, _DTYPES[dy.dtype], vocab, cols, scale, gp, ldg,
                                 bool(add), wsp, need), dy.get_device())
    _written(given)
    return out


def _grads(gs, name):
    """(tensors, their count, pointers, sizes) of one gradient or a list of them: one dtype, one device, contiguous."""
    gs = (gs,) if isinstance(gs, torch.Tensor) else gs
    count = len(gs)
    if not count:
        raise ValueError(f"need at least one of {name}")
    dt, index = gs[0].dtype, gs[0].get_device()
    if dt not in _DTYPES:
        raise TypeError(f"{name} have dtype {dt}, expected float32, bfloat16 or float16")
    open_level = _forward_ad._current_level >= 0
    for r, g in enumerate(gs):
        if g.dtype != dt or g.get_device() != index or not g.is_cuda or not g.is_contiguous() or \
                g.requires_grad or open_level:
            _refuse(g, f"{name}[{r}]", dt, gs[0].device)
    return gs, count, (ctypes.c_void_p * count)(*[g.data_ptr() for g in gs]), \
        (ctypes.c_int64 * count)(*[g.numel() for g in gs])


def _refuse(g, name, dtype, device):
    if not g.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (there is no CPU path)")
    if g.dtype != dtype:
        raise TypeError(f"{name} has dtype {g.dtype}, expected {dtype}")
    if g.device != device:
        raise ValueError(f"{name} is on {g.device}, the call's other tensors on {device}")
    if not g.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    _unfollowed(g, name)


def _scalar(t, name, beside):
    """(tensor, pointer) of a float32 scalar on the device, a new one where none is given."""
    if t is None:
        t = torch.empty((), dtype=torch.float32, device=beside.device)
    return t, _row_values(t, name, 1, beside)


@functools.lru_cache(maxsize=64)
def _grad_workspace(count):
    return _lib.demo_grad_workspace(count)


def grad_norm(gs, *, out=None, workspace=None, stream=None):
    """The norm over all elements of a gradient, or of a list of them (one dtype, contiguous), as a float32
    scalar on the device (demo_grad_norm); ``out`` receives it."""
    if stream is None and workspace is None:
        r = _bind.grad_norm(gs, out)
        if r.__class__ is int:
            _refused(r, "demo_grad_norm")
        if r is not NotImplemented:
            return r
    if stream is not None:
        first = gs if isinstance(gs, torch.Tensor) else gs[0]
        return _on_stream(stream, first.device, grad_norm, gs, out=out, workspace=workspace)
    gs, count, ptrs, sizes = _grads(gs, "gradients")
    given = out
    out, op = _scalar(out, "out", gs[0])
    workspace, wsp, need = _workspace(workspace, _grad_workspace(count), gs[0])
    _run("demo_grad_norm", (count, ptrs, sizes, _DTYPES[gs[0].dtype], op, wsp, need), gs[0].get_device())
    _written(given)
    return out


def clip_grads(gs, max_norm, *, norm=None, out=None, workspace=None, stream=None):
    """Scales a gradient, or a list of them (one dtype, contiguous), to a norm of ``max_norm`` at most
    (demo_clip_grads); returns the norm before, a float32 scalar on the device.  Nothing waits for the device.

    ``norm``  the norm to clip by, where it is not that of ``gs`` alone (gradients in several shards); it is
              computed otherwise
    ``out``   tensors of the same sizes to write, in the gradients' dtype or float32; in place otherwise
    A norm that is not finite scales nothing.
    """
    if stream is None and workspace is None:
        r = _bind.clip_grads(gs, max_norm, norm, out)
        if r.__class__ is int:
            _refused(r, "demo_clip_grads")
        if r is not NotImplemented:
            return r
    if stream is not None:
        first = gs if isinstance(gs, torch.Tensor) else gs[0]
        return _on_stream(stream, first.device, clip_grads, gs, max_norm, norm=norm, out=out, workspace=workspace)
    gs, count, ptrs, sizes = _grads(gs, "gradients")
    outs, odt = None, gs[0].dtype
    if out is not None:
        out, n, outs, to = _grads(out, "outs")
        odt = out[0].dtype
        if n != count or any(a != b for a, b in zip(sizes, to)):
            raise ValueError("out must hold a tensor of the same size for each gradient")
        if out[0].get_device() != gs[0].get_device():
            raise ValueError(f"out is on {out[0].device}, the gradients on {gs[0].device}")
    given = norm is not None
    norm, normp = _scalar(norm, "norm", gs[0])
    workspace, wsp, need = _workspace(workspace, 0 if given else _grad_workspace(count), gs[0])
    _run("demo_clip_grads", (count, ptrs, sizes, _DTYPES[gs[0].dtype], outs, _DTYPES[odt], max_norm, normp, given, wsp, need),
         gs[0].get_device())
    _wrote(list(gs if out is None else out))
    return norm
