"""The expert path's operators on torch CUDA tensors (``include/moe_ops.h``).

Used together they make an expert path of one's own::

    r = F.sort_tokens(ids, n_experts)                     # ids int32 [T, k]
    q = F.fp4_quantize(x, "nvfp4")                        # a scale per token
    xs = F.FP4Tensor(*(F.dispatch(t, r["inv"]) for t in (q.codes, q.scales)),
                     F.dispatch(q.global_scale[:, None], r["inv"])[:, 0], q.fmt)
    h = activation(F.fp4_matmul(xs, w_in, r["offsets"]))
    ys = F.fp4_matmul(F.fp4_quantize(h, "nvfp4"), w_out, r["offsets"])
    y = F.combine(ys, r["inv"], gates)

Every call checks its arguments, enqueues kernels on the current stream of the
tensors' device (or on ``stream``) and returns; a refused argument raises
:class:`MoEError`.  ``out`` takes the result in the caller's own tensor; rows
that a call does not write (see the header) are then left as they were, and are
uninitialised in a result that the call allocates.  The gradients are calls of
their own: nothing here records an autograd graph.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from ._lib import MoEError, check, lib

_DTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2, torch.uint8: 3}
_BLOCK = {"mxfp4": 32, "nvfp4": 16}
_U8, _I32, _F32 = torch.uint8, torch.int32, torch.float32
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
try:   # the allocation alone, without torch.empty's argument parsing (2.5 us of a small call's 10)
    from torch._C._dynamo.guards import _empty_strided_cuda as _empty_strided
except ImportError:
    def _empty_strided(size, stride, dtype):
        return torch.empty_strided(size, stride, dtype=dtype, device="cuda")


def _int32(fn, what, n):
    """The C entry points take sizes as int32, which ctypes would cut silently."""
    if n > 0x7FFFFFFF:
        _bad(f"{fn}: {what} = {n} must be below 2^31")


def _new(n, cols, dtype):
    """An uninitialised contiguous tensor [n, cols] on the current device."""
    return _empty_strided((n, cols), (cols, 1), dtype)


class FP4Tensor(NamedTuple):
    """FP4 values in checkpoint layout: ``codes`` uint8 [..., K/2], ``scales`` uint8
    [..., K/32] (mxfp4) or [..., K/16] (nvfp4), ``global_scale`` fp32 (nvfp4, else
    None) with one value for each row, or for each matrix of a 3-D tensor."""
    codes: torch.Tensor
    scales: torch.Tensor
    global_scale: Optional[torch.Tensor]
    fmt: str


def _bad(what):
    raise MoEError(1, what)


def _elsewhere(fn, t, stream, used, *args):
    """fn(*args) with the device of t current and, if given, on `stream`: what the
    call allocates belongs to that stream, and what it uses is kept for it."""
    dev = t.device
    if dev.type != "cuda":
        _bad(f"{fn.__name__}: the tensors must be CUDA tensors, not on {dev}")
    with torch.cuda.device(dev):
        if stream is None:
            return fn(*args)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, dev) if stream else torch.cuda.default_stream(dev)
        if stream.device != dev:
            _bad(f"{fn.__name__}: the stream is of {stream.device}, the tensors of {dev}")
        with torch.cuda.stream(stream):
            got = fn(*args)
            for t in used:
                if t is not None:
                    t.record_stream(stream)
            return got


def _same(fn, dev, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != dev:
            _bad(f"{fn}: tensors on cuda:{dev} and {t.device}")


def _ld(fn, name, t, rows, cols):
    """Row stride of a 2-D tensor with contiguous rows."""
    if t.is_contiguous():
        return cols
    ld, inner = t.stride()
    if cols > 1 and inner != 1:
        _bad(f"{fn}: the rows of {name} must be contiguous")
    return ld if rows > 1 else cols


def _float(fn, name, t):
    d = _DTYPE.get(t.dtype, 3)
    if d == 3:
        _bad(f"{fn}: {name} must be float32, bfloat16 or float16, not {t.dtype}")
    return d


def _want(fn, name, t, dtype, shape):
    """A contiguous tensor of this type and shape."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _bad(f"{fn}: {name} must be contiguous {dtype} {list(shape)}, not {t.dtype} {list(t.shape)}")


# ------------------------------------------------------------------------ FP4
def _fp4(fn, name, q, dev):
    """(leading shape, K, fmt code) of an FP4Tensor whose parts fit together."""
    codes, scales, g, fmt = q
    block = _BLOCK.get(fmt)
    if block is None:
        _bad(f"{fn}: format {fmt!r} is not 'mxfp4' or 'nvfp4'")
    shape = codes.shape
    K = 2 * shape[-1]
    if codes.dtype is not _U8 or not codes.is_contiguous():
        _bad(f"{fn}: {name}.codes must be contiguous uint8")
    if K % 32:
        _bad(f"{fn}: K = {K} of {name} is not a multiple of 32")
    lead = shape[:-1]
    if scales.dtype is not _U8 or not scales.is_contiguous() or scales.shape != (*lead, K // block):
        _want(fn, name + ".scales", scales, _U8, (*lead, K // block))
    if (g is None) != (fmt == "mxfp4"):
        _bad(f"{fn}: {name}.global_scale belongs to nvfp4, and to it alone")
    _same(fn, dev, codes, scales, g)
    return lead, K, 0 if g is None else 1


def fp4_quantize(x, fmt="mxfp4", rows_per_scale=None, out=None, stream=None):
    """Quantise x [rows, K] or [matrices, rows, K] (float32, bfloat16, float16) to an
    :class:`FP4Tensor`.  nvfp4 has one fp32 scale for each ``rows_per_scale`` rows:
    by default one per row of a 2-D tensor, one per matrix of a 3-D one."""
    fn = "fp4_quantize"
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(fp4_quantize, x, stream, (x,) if out is None else (x, *out[:3]), x, fmt, rows_per_scale, out)
    block = _BLOCK.get(fmt)
    if block is None:
        _bad(f"{fn}: format {fmt!r} is not 'mxfp4' or 'nvfp4'")
    shape, x2 = x.shape, x
    if len(shape) == 3:
        try:
            x2 = x.view(shape[0] * shape[1], shape[2])
        except RuntimeError:
            _bad(f"{fn}: the matrices of x must follow one another at one row stride")
        if rows_per_scale is None:
            rows_per_scale = max(1, shape[1])
    elif len(shape) != 2:
        _bad(f"{fn}: x must have two or three axes, not {len(shape)}")
    n, K = x2.shape
    per = 1 if rows_per_scale is None else int(rows_per_scale)
    if per < 1 or n % per:
        _bad(f"{fn}: {n} rows are not a multiple of rows_per_scale = {per}")
    if K < 32 or K % 32:
        _bad(f"{fn}: K = {K} is not a multiple of 32")
    nv, half, nsf = block == 16, K // 2, K // block
    if out is None:
        if len(shape) == 2:
            codes, scales = _new(n, half, _U8), _new(n, nsf, _U8)
        else:
            codes, scales = _new(n, half, _U8).view(*shape[:2], half), _new(n, nsf, _U8).view(*shape[:2], nsf)
        g = _empty_strided((n // per,), (1,), _F32) if nv else None
        out = FP4Tensor(codes, scales, g, fmt)
    else:
        if out.fmt != fmt or _fp4(fn, "out", out, dev)[:2] != (shape[:-1], K):
            _bad(f"{fn}: out is of another format or shape")
        codes, scales, g = out.codes, out.scales, out.global_scale
        if nv:
            _want(fn, "out.global_scale", g, _F32, (n // per,))
    status = lib().moe_fp4_quantize(x2.data_ptr(), _float(fn, "x", x), n, K, _ld(fn, "x", x2, n, K), 1 if nv else 0, per,
                                 codes.data_ptr(), scales.data_ptr(), g.data_ptr() if nv else None,
                                 _raw_stream(dev))
    if status:
        check(status)
    return out


def fp4_dequantize(q, dtype=torch.float32, out=None, stream=None):
    """The values of an :class:`FP4Tensor`, rounded to ``dtype`` (float32 is exact)."""
    fn = "fp4_dequantize"
    codes, scales, g, _ = q
    dev = codes.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(fp4_dequantize, codes, stream, (codes, scales, g, out), q, dtype, out)
    lead, K, fmt = _fp4(fn, "q", q, dev)
    n = lead[0] if len(lead) == 1 else lead.numel()
    per = 1
    if g is not None:
        if g.dtype is not _F32 or not g.is_contiguous():
            _bad(f"{fn}: q.global_scale must be contiguous float32, not {g.dtype}")
        groups = g.numel()
        if n and (not groups or n % groups):
            _bad(f"{fn}: {groups} global scales do not divide {n} rows")
        per = max(1, n // max(1, groups))
    if out is None:
        o2 = _new(n, K, dtype)
        out = o2 if len(lead) == 1 else o2.view(*lead, K)
    else:
        if out.shape != (*lead, K) or (len(lead) != 1 and not out.is_contiguous()):
            _bad(f"{fn}: out must be {[*lead, K]}, contiguous if it has three axes, not {list(out.shape)}")
        _same(fn, dev, out)
        o2 = out if len(lead) == 1 else out.view(n, K)
    status = lib().moe_fp4_dequantize(codes.data_ptr(), scales.data_ptr(), None if g is None else g.data_ptr(), fmt, n, K,
                                   per, o2.data_ptr(), _float(fn, "out", o2), _ld(fn, "out", o2, n, K),
                                   _raw_stream(dev))
    if status:
        check(status)
    return out


def fp4_matmul(x, w, offsets=None, out_dtype=torch.bfloat16, out=None, stream=None):
    """x [rows, K] times the transpose of w [N, K] or, by groups of rows, of w [groups, N, K].

    Both are :class:`FP4Tensor` of one format (nvfp4: a global scale per row of x
    and per matrix of w).  ``offsets`` int32 [groups + 1] gives each group's rows
    (``sort_tokens`` writes it); without it w has one matrix and takes every row.
    Rows outside the groups are not written.  ``out`` takes the result in its own
    type."""
    fn = "fp4_matmul"
    xc, xs, xg, _ = x
    wc, ws, wg, _ = w
    dev = xc.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(fp4_matmul, xc, stream, (xc, xs, xg, wc, ws, wg, offsets, out), x, w, offsets, out_dtype, out)
    lead, K, fmt = _fp4(fn, "x", x, dev)
    wlead, wK, wfmt = _fp4(fn, "w", w, dev)
    if len(lead) != 1 or len(wlead) not in (1, 2) or wK != K or wfmt != fmt:
        _bad(f"{fn}: x {list(xc.shape)} {x.fmt} and w {list(wc.shape)} {w.fmt} do not multiply")
    n, N = lead[0], wlead[-1]
    if n > 0x7FFFFFFF or N > 0x7FFFFFFF or K > 0x7FFFFFFF:
        _int32(fn, "a size", max(n, N, K))
    groups = wlead[0] if len(wlead) == 2 else 1
    if fmt:
        _want(fn, "x.global_scale", xg, _F32, (n,))
        _want(fn, "w.global_scale", wg, _F32, (groups,))
    if offsets is not None:
        _want(fn, "offsets", offsets, _I32, (groups + 1,))
        _same(fn, dev, offsets)
    elif groups != 1:
        _bad(f"{fn}: {groups} groups need offsets")
    if out is None:
        out = _new(n, N, out_dtype)
    else:
        if out.shape != (n, N):
            _bad(f"{fn}: out must be [{n}, {N}], not {list(out.shape)}")
        _same(fn, dev, out)
    status = lib().moe_fp4_matmul(xc.data_ptr(), xs.data_ptr(), xg.data_ptr() if fmt else None, n, wc.data_ptr(),
                               ws.data_ptr(), wg.data_ptr() if fmt else None, groups, N, K, fmt,
                               None if offsets is None else offsets.data_ptr(), out.data_ptr(),
                               _float(fn, "out", out), _ld(fn, "out", out, n, N), _raw_stream(dev))
    if status:
        check(status)
    return out


# ----------------------------------------------------------------- expert rows
def sort_tokens(ids, n_experts, stream=None):
    """Sort the pairs of ids int32 [T, k] by expert (stable).  Returns counts [E],
    offsets [E + 1], perm [T * k] (position -> pair, -1 behind the last) and inv
    [T, k] (pair -> position, -1 where the id is outside [0, E): a dropped pair)."""
    dev = ids.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(sort_tokens, ids, stream, (ids,), ids, n_experts)
    shape = ids.shape
    if len(shape) != 2 or ids.dtype is not _I32 or not ids.is_contiguous():
        _bad(f"sort_tokens: ids must be contiguous int32 [T, k], not {ids.dtype} {list(shape)}")
    T, k = shape
    E = int(n_experts)
    if T * k > 0x7FFFFFFF:
        _int32("sort_tokens", "T * k", T * k)
    if not 1 <= E <= 1024:
        _bad(f"sort_tokens: {E} experts: 1 to 1024 are supported")
    counts, offsets = _empty_strided((E,), (1,), _I32), _empty_strided((E + 1,), (1,), _I32)
    perm, inv = _empty_strided((T * k,), (1,), _I32), _new(T, k, _I32)
    status = lib().moe_sort_tokens(ids.data_ptr(), T, k, E, counts.data_ptr(), offsets.data_ptr(), perm.data_ptr(),
                                inv.data_ptr(), _raw_stream(dev))
    if status:
        check(status)
    return {"counts": counts, "offsets": offsets, "perm": perm, "inv": inv}


def _pairs(fn, inv, T, dev, gates=None):
    """k of inv [T, k], which has to be on this device, as the gates have."""
    shape = inv.shape
    if len(shape) != 2 or inv.dtype is not _I32 or not inv.is_contiguous() or (T is not None and shape[0] != T):
        _bad(f"{fn}: inv must be contiguous int32 [{'T' if T is None else T}, k], not {inv.dtype} {list(shape)}")
    if shape[0] * shape[1] > 0x7FFFFFFF:
        _int32(fn, "T * k", shape[0] * shape[1])
    if gates is not None:
        _want(fn, "gates", gates, _F32, shape)
    _same(fn, dev, inv, gates)
    return shape


def _two(fn, name, t):
    shape = t.shape
    if len(shape) != 2:
        _bad(f"{fn}: {name} must have two axes, not {len(shape)}")
    if shape[0] > 0x7FFFFFFF or shape[1] > 0x7FFFFFFF:
        _int32(fn, f"an axis of {name}", max(shape))
    return shape


def _out(fn, out, dtype, n, cols, dev):
    """`out` if it is [n, cols] of this type (any, if dtype is None) on this device."""
    if out.shape != (n, cols) or (dtype is not None and out.dtype is not dtype):
        _bad(f"{fn}: out must be {dtype} [{n}, {cols}], not {out.dtype} {list(out.shape)}")
    _same(fn, dev, out)
    return out


def dispatch(x, inv, rows=None, out=None, stream=None):
    """xs[inv[t, j]] = x[t].  x [T, H]: float32, bfloat16, float16 or uint8 (codes,
    scales); xs [rows, H], rows = T * k unless given (or out's); positions from
    ``rows`` on are dropped, rows that no pair names are not written."""
    fn = "dispatch"
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(dispatch, x, stream, (x, inv, out), x, inv, rows, out)
    T, H = _two(fn, "x", x)
    k = _pairs(fn, inv, T, dev)[1]
    dtype = x.dtype
    dt = _DTYPE.get(dtype)
    if dt is None:
        _bad(f"{fn}: x must be float32, bfloat16, float16 or uint8, not {dtype}")
    if out is None:
        rows = T * k if rows is None else int(rows)
        if not 0 <= rows <= 0x7FFFFFFF:
            _bad(f"{fn}: rows = {rows} must be 0 to 2^31 - 1")
        out = _new(rows, H, dtype)
    else:
        rows = out.shape[0] if rows is None else rows
        _out(fn, out, dtype, rows, H, dev)
    status = lib().moe_dispatch(x.data_ptr(), dt, T, k, H, _ld(fn, "x", x, T, H), inv.data_ptr(), rows, out.data_ptr(),
                             _ld(fn, "out", out, rows, H), _raw_stream(dev))
    if status:
        check(status)
    return out


def dispatch_backward(dxs, inv, out=None, stream=None):
    """Gradient of :func:`dispatch`: dx[t] = sum over t's pairs of dxs[inv[t, j]] (fp32, rounded once)."""
    fn = "dispatch_backward"
    dev = dxs.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(dispatch_backward, dxs, stream, (dxs, inv, out), dxs, inv, out)
    rows, H = _two(fn, "dxs", dxs)
    T, k = _pairs(fn, inv, None, dev)
    dt = _float(fn, "dxs", dxs)
    out = _new(T, H, dxs.dtype) if out is None else _out(fn, out, dxs.dtype, T, H, dev)
    status = lib().moe_dispatch_backward(dxs.data_ptr(), dt, rows, T, k, H, _ld(fn, "dxs", dxs, rows, H), inv.data_ptr(),
                                      out.data_ptr(), _ld(fn, "out", out, T, H), _raw_stream(dev))
    if status:
        check(status)
    return out


def combine(ys, inv, gates=None, out_dtype=None, out=None, stream=None):
    """y[t] = sum over t's pairs of gates[t, j] * ys[inv[t, j]] (fp32, rounded once to
    ``out_dtype``, by default ys's).  gates fp32 [T, k], or None for ones."""
    fn = "combine"
    dev = ys.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(combine, ys, stream, (ys, inv, gates, out), ys, inv, gates, out_dtype, out)
    rows, H = _two(fn, "ys", ys)
    T, k = _pairs(fn, inv, None, dev, gates)
    out = _new(T, H, out_dtype or ys.dtype) if out is None else _out(fn, out, out_dtype, T, H, dev)
    status = lib().moe_combine(ys.data_ptr(), _float(fn, "ys", ys), rows, T, k, H, _ld(fn, "ys", ys, rows, H),
                            inv.data_ptr(), None if gates is None else gates.data_ptr(), out.data_ptr(),
                            _float(fn, "out", out), _ld(fn, "out", out, T, H), _raw_stream(dev))
    if status:
        check(status)
    return out


def combine_backward(dy, ys, inv, gates=None, out=None, stream=None):
    """Gradients of :func:`combine`: (dys, dgates).  dys[inv[t, j]] = gates[t, j] * dy[t]
    in ys's type (``out`` takes it; rows that no pair names are not written);
    dgates[t, j] = <dy[t], ys[inv[t, j]]> fp32 [T, k], 0 for a dropped pair."""
    fn = "combine_backward"
    dev = dy.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(combine_backward, dy, stream, (dy, ys, inv, gates, out), dy, ys, inv, gates, out)
    T, H = _two(fn, "dy", dy)
    rows, Hs = _two(fn, "ys", ys)
    if Hs != H:
        _bad(f"{fn}: dy {[T, H]} and ys {[rows, Hs]} do not belong together")
    _same(fn, dev, ys)
    k = _pairs(fn, inv, T, dev, gates)[1]
    out = _new(rows, H, ys.dtype) if out is None else _out(fn, out, ys.dtype, rows, H, dev)
    dgates = _new(T, k, _F32)
    status = lib().moe_combine_backward(dy.data_ptr(), _float(fn, "dy", dy), _ld(fn, "dy", dy, T, H), ys.data_ptr(),
                                     _float(fn, "ys", ys), _ld(fn, "ys", ys, rows, H), rows, T, k, H, inv.data_ptr(),
                                     None if gates is None else gates.data_ptr(), out.data_ptr(),
                                     _ld(fn, "out", out, rows, H), dgates.data_ptr(), _raw_stream(dev))
    if status:
        check(status)
    return out, dgates
