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

from ._lib import FMT, MoEError, check, lib

_DTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2, torch.uint8: 3}
_BLOCK = {"mxfp4": 32, "nvfp4": 16}
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


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


def _elsewhere(fn, dev, stream, tensors, *args):
    """fn(*args) with the tensors' device current and, if given, on `stream`:
    what the call allocates belongs to that stream, and what it uses is kept for it."""
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
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
            return got


def _same_device(fn, dev, *tensors):
    for t in tensors:
        if t is not None and t.device != dev:
            _bad(f"{fn}: tensors on {dev} and {t.device}")


def _ld(fn, name, t):
    """Row stride of a 2-D tensor with contiguous rows."""
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        _bad(f"{fn}: the rows of {name} must be contiguous")
    return t.stride(0) if rows > 1 else max(cols, 1)


def _float(fn, name, t):
    d = _DTYPE.get(t.dtype, 3)
    if d == 3:
        _bad(f"{fn}: {name} must be float32, bfloat16 or float16, not {t.dtype}")
    return d


def _ptr(t):
    return None if t is None else t.data_ptr()


def _contiguous(fn, name, t, dtype, shape):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _bad(f"{fn}: {name} must be contiguous {dtype} {list(shape)}, not {t.dtype} {list(t.shape)}")


# ------------------------------------------------------------------------ FP4
def _fp4(fn, name, q):
    """(leading shape, K, fmt code) of an FP4Tensor whose parts fit together."""
    if q.fmt not in _BLOCK:
        _bad(f"{fn}: format {q.fmt!r} is not 'mxfp4' or 'nvfp4'")
    lead, K = q.codes.shape[:-1], 2 * q.codes.shape[-1]
    _contiguous(fn, name + ".codes", q.codes, torch.uint8, q.codes.shape)
    _contiguous(fn, name + ".scales", q.scales, torch.uint8, lead + (K // _BLOCK[q.fmt],))
    if (q.global_scale is None) != (q.fmt == "mxfp4"):
        _bad(f"{fn}: {name}.global_scale belongs to nvfp4, and to it alone")
    if K % 32:
        _bad(f"{fn}: K = {K} of {name} is not a multiple of 32")
    return lead, K, FMT[q.fmt]


def fp4_quantize(x, fmt="mxfp4", rows_per_scale=None, out=None, stream=None):
    """Quantise x [rows, K] or [matrices, rows, K] (float32, bfloat16, float16) to an
    :class:`FP4Tensor`.  nvfp4 has one fp32 scale for each ``rows_per_scale`` rows:
    by default one per row of a 2-D tensor, one per matrix of a 3-D one."""
    dev = x.device
    if stream is not None or dev.type != "cuda" or dev.index != _current_device():
        used = (x,) if out is None else (x, *out[:3])
        return _elsewhere(fp4_quantize, dev, stream, used, x, fmt, rows_per_scale, out)
    dt = _float("fp4_quantize", "x", x)
    if fmt not in _BLOCK:
        _bad(f"fp4_quantize: format {fmt!r} is not 'mxfp4' or 'nvfp4'")
    lead = x.shape[:-1]
    if x.dim() == 3:
        if rows_per_scale is None:
            rows_per_scale = max(1, x.shape[1])
        if x.shape[0] > 1 and x.stride(0) != x.shape[1] * x.stride(1):
            _bad("fp4_quantize: the matrices of x must follow one another at the row stride")
        x2 = x.flatten(0, 1)
    elif x.dim() == 2:
        x2 = x
    else:
        _bad(f"fp4_quantize: x must have two or three axes, not {x.dim()}")
    n, K = x2.shape
    per = 1 if rows_per_scale is None else int(rows_per_scale)
    if per < 1 or n % per:
        _bad(f"fp4_quantize: {n} rows are not a multiple of rows_per_scale = {per}")
    if K < 32 or K % 32:
        _bad(f"fp4_quantize: K = {K} is not a multiple of 32")
    nv = fmt == "nvfp4"
    if out is None:
        out = FP4Tensor(torch.empty(lead + (K // 2,), dtype=torch.uint8, device=dev),
                        torch.empty(lead + (K // _BLOCK[fmt],), dtype=torch.uint8, device=dev),
                        torch.empty(n // per, dtype=torch.float32, device=dev) if nv else None, fmt)
    else:
        _same_device("fp4_quantize", dev, *out[:3])
        if out.fmt != fmt or _fp4("fp4_quantize", "out", out)[:2] != (lead, K):
            _bad("fp4_quantize: out is of another format or shape")
        if nv:
            _contiguous("fp4_quantize", "out.global_scale", out.global_scale, torch.float32, (n // per,))
    check(lib().moe_fp4_quantize(x2.data_ptr(), dt, n, K, _ld("fp4_quantize", "x", x2), FMT[fmt], per,
                                 out.codes.data_ptr(), out.scales.data_ptr(), _ptr(out.global_scale),
                                 _raw_stream(dev.index)))
    return out


def fp4_dequantize(q, dtype=torch.float32, out=None, stream=None):
    """The values of an :class:`FP4Tensor`, rounded to ``dtype`` (float32 is exact)."""
    dev = q.codes.device
    if stream is not None or dev.type != "cuda" or dev.index != _current_device():
        return _elsewhere(fp4_dequantize, dev, stream, (*q[:3], out), q, dtype, out)
    fn = "fp4_dequantize"
    lead, K, fmt = _fp4(fn, "q", q)
    n = q.codes.shape[:-1].numel()
    per = 1
    if q.global_scale is not None:
        g = q.global_scale.numel()
        _contiguous(fn, "q.global_scale", q.global_scale, torch.float32, q.global_scale.shape)
        if n and (not g or n % g):
            _bad(f"{fn}: {g} global scales do not divide {n} rows")
        per = max(1, n // max(1, g))
    if out is None:
        out = torch.empty(lead + (K,), dtype=dtype, device=dev)
    elif out.shape != lead + (K,):
        _bad(f"{fn}: out must be {list(lead) + [K]}, not {list(out.shape)}")
    _same_device(fn, dev, q.scales, q.global_scale, out)
    o2 = out if out.dim() == 2 else out.view(n, K)
    check(lib().moe_fp4_dequantize(q.codes.data_ptr(), q.scales.data_ptr(), _ptr(q.global_scale), fmt, n, K, per,
                                   o2.data_ptr(), _float(fn, "out", out), _ld(fn, "out", o2),
                                   _raw_stream(dev.index)))
    return out


def fp4_matmul(x, w, offsets=None, out_dtype=torch.bfloat16, out=None, stream=None):
    """x [rows, K] times the transpose of w [N, K] or, by groups of rows, of w [groups, N, K].

    Both are :class:`FP4Tensor` of one format (nvfp4: a global scale per row of x
    and per matrix of w).  ``offsets`` int32 [groups + 1] gives each group's rows
    (``sort_tokens`` writes it); without it w has one matrix and takes every row.
    Rows outside the groups are not written."""
    xc = x.codes
    dev = xc.device
    if stream is not None or dev.type != "cuda" or dev.index != _current_device():
        return _elsewhere(fp4_matmul, dev, stream, (*x[:3], *w[:3], offsets, out), x, w, offsets, out_dtype, out)
    fn = "fp4_matmul"
    lead, K, fmt = _fp4(fn, "x", x)
    wlead, wK, wfmt = _fp4(fn, "w", w)
    if len(lead) != 1 or len(wlead) not in (1, 2) or wK != K or wfmt != fmt:
        _bad(f"{fn}: x {list(xc.shape)} {x.fmt} and w {list(w.codes.shape)} {w.fmt} do not multiply")
    n, N = lead[0], wlead[-1]
    groups = wlead[0] if len(wlead) == 2 else 1
    if x.global_scale is not None:
        _contiguous(fn, "x.global_scale", x.global_scale, torch.float32, (n,))
        _contiguous(fn, "w.global_scale", w.global_scale, torch.float32, (groups,))
    if offsets is not None:
        _contiguous(fn, "offsets", offsets, torch.int32, (groups + 1,))
    elif groups != 1:
        _bad(f"{fn}: {groups} groups need offsets")
    if out is None:
        out = torch.empty((n, N), dtype=out_dtype, device=dev)
    elif out.shape != (n, N):
        _bad(f"{fn}: out must be [{n}, {N}], not {list(out.shape)}")
    _same_device(fn, dev, x.scales, x.global_scale, w.codes, w.scales, w.global_scale, offsets, out)
    check(lib().moe_fp4_matmul(xc.data_ptr(), x.scales.data_ptr(), _ptr(x.global_scale), n, w.codes.data_ptr(),
                               w.scales.data_ptr(), _ptr(w.global_scale), groups, N, K, fmt, _ptr(offsets),
                               out.data_ptr(), _float(fn, "out", out), _ld(fn, "out", out), _raw_stream(dev.index)))
    return out


# ----------------------------------------------------------------- expert rows
def sort_tokens(ids, n_experts, stream=None):
    """Sort the pairs of ids int32 [T, k] by expert (stable).  Returns counts [E],
    offsets [E + 1], perm [T * k] (position -> pair, -1 behind the last) and inv
    [T, k] (pair -> position, -1 where the id is outside [0, E): a dropped pair)."""
    dev = ids.device
    if stream is not None or dev.type != "cuda" or dev.index != _current_device():
        return _elsewhere(sort_tokens, dev, stream, (ids,), ids, n_experts)
    if ids.dim() != 2 or ids.dtype is not torch.int32 or not ids.is_contiguous():
        _bad(f"sort_tokens: ids must be contiguous int32 [T, k], not {ids.dtype} {list(ids.shape)}")
    T, k = ids.shape
    E, n = int(n_experts), T * k
    if not 1 <= E <= 1024:
        _bad(f"sort_tokens: {E} experts: 1 to 1024 are supported")
    counts, offsets, perm, inv = torch.empty(2 * E + 1 + 2 * n, dtype=torch.int32, device=dev).split((E, E + 1, n, n))
    check(lib().moe_sort_tokens(ids.data_ptr(), T, k, E, counts.data_ptr(), offsets.data_ptr(), perm.data_ptr(),
                                inv.data_ptr(), _raw_stream(dev.index)))
    return {"counts": counts, "offsets": offsets, "perm": perm, "inv": inv.view(T, k)}


def _inv(fn, inv, T, dev):
    if inv.dim() != 2 or inv.dtype is not torch.int32 or not inv.is_contiguous() or inv.shape[0] != T:
        _bad(f"{fn}: inv must be contiguous int32 [{T}, k], not {inv.dtype} {list(inv.shape)}")
    if inv.device != dev:
        _bad(f"{fn}: tensors on {dev} and {inv.device}")
    return inv.shape[1]


def _two(fn, name, t):
    if t.dim() != 2:
        _bad(f"{fn}: {name} must have two axes, not {t.dim()}")
    return t.shape


def _gates(fn, gates, T, k, dev):
    if gates is not None:
        _contiguous(fn, "gates", gates, torch.float32, (T, k))
        if gates.device != dev:
            _bad(f"{fn}: tensors on {dev} and {gates.device}")


def dispatch(x, inv, rows=None, out=None, stream=None):
    """xs[inv[t, j]] = x[t].  x [T, H]: float32, bfloat16, float16 or uint8 (codes,
    scales); xs [rows, H], rows = T * k unless given (or out's); positions from
    ``rows`` on are dropped, rows that no pair names are not written."""
    dev = x.device
    if stream is not None or dev.type != "cuda" or dev.index != _current_device():
        return _elsewhere(dispatch, dev, stream, (x, inv, out), x, inv, rows, out)
    T, H = _two("dispatch", "x", x)
    k = _inv("dispatch", inv, T, dev)
    dt = _DTYPE.get(x.dtype)
    if dt is None:
        _bad(f"dispatch: x must be float32, bfloat16, float16 or uint8, not {x.dtype}")
    if out is None:
        out = torch.empty((T * k if rows is None else rows, H), dtype=x.dtype, device=dev)
    elif out.dim() != 2 or out.dtype is not x.dtype or out.shape[1] != H or out.device != dev or \
            rows not in (None, out.shape[0]):
        _bad(f"dispatch: out must be {x.dtype} [rows, {H}] on {dev}, not {out.dtype} {list(out.shape)} on {out.device}")
    check(lib().moe_dispatch(x.data_ptr(), dt, T, k, H, _ld("dispatch", "x", x), inv.data_ptr(), out.shape[0],
                             out.data_ptr(), _ld("dispatch", "out", out), _raw_stream(dev.index)))
    return out


def dispatch_backward(dxs, inv, out=None, stream=None):
    """Gradient of :func:`dispatch`: dx[t] = sum over t's pairs of dxs[inv[t, j]] (fp32, rounded once)."""
    dev = dxs.device
    if stream is not None or dev.type != "cuda" or dev.index != _current_device():
        return _elsewhere(dispatch_backward, dev, stream, (dxs, inv, out), dxs, inv, out)
    fn = "dispatch_backward"
    rows, H = _two(fn, "dxs", dxs)
    T = inv.shape[0]
    k = _inv(fn, inv, T, dev)
    if out is None:
        out = torch.empty((T, H), dtype=dxs.dtype, device=dev)
    elif out.shape != (T, H) or out.dtype is not dxs.dtype or out.device != dev:
        _bad(f"{fn}: out must be {dxs.dtype} [{T}, {H}] on {dev}")
    check(lib().moe_dispatch_backward(dxs.data_ptr(), _float(fn, "dxs", dxs), rows, T, k, H, _ld(fn, "dxs", dxs),
                                      inv.data_ptr(), out.data_ptr(), _ld(fn, "out", out), _raw_stream(dev.index)))
    return out


def combine(ys, inv, gates=None, out_dtype=None, out=None, stream=None):
    """y[t] = sum over t's pairs of gates[t, j] * ys[inv[t, j]] (fp32, rounded once to
    ``out_dtype``, by default ys's).  gates fp32 [T, k], or None for ones."""
    dev = ys.device
    if stream is not None or dev.type != "cuda" or dev.index != _current_device():
        return _elsewhere(combine, dev, stream, (ys, inv, gates, out), ys, inv, gates, out_dtype, out)
    rows, H = _two("combine", "ys", ys)
    T = inv.shape[0]
    k = _inv("combine", inv, T, dev)
    _gates("combine", gates, T, k, dev)
    if out is None:
        out = torch.empty((T, H), dtype=out_dtype or ys.dtype, device=dev)
    elif out.shape != (T, H) or out.device != dev or out_dtype not in (None, out.dtype):
        _bad(f"combine: out must be {out_dtype or ys.dtype} [{T}, {H}] on {dev}")
    check(lib().moe_combine(ys.data_ptr(), _float("combine", "ys", ys), rows, T, k, H, _ld("combine", "ys", ys),
                            inv.data_ptr(), _ptr(gates), out.data_ptr(), _float("combine", "out", out),
                            _ld("combine", "out", out), _raw_stream(dev.index)))
    return out


def combine_backward(dy, ys, inv, gates=None, out=None, stream=None):
    """Gradients of :func:`combine`: (dys, dgates).  dys[inv[t, j]] = gates[t, j] * dy[t]
    in ys's type (``out`` takes it; rows that no pair names are not written);
    dgates[t, j] = <dy[t], ys[inv[t, j]]> fp32 [T, k], 0 for a dropped pair."""
    dev = dy.device
    if stream is not None or dev.type != "cuda" or dev.index != _current_device():
        return _elsewhere(combine_backward, dev, stream, (dy, ys, inv, gates, out), dy, ys, inv, gates, out)
    fn = "combine_backward"
    T, H = _two(fn, "dy", dy)
    rows, Hs = _two(fn, "ys", ys)
    if Hs != H or ys.device != dev:
        _bad(f"{fn}: dy {list(dy.shape)} on {dev} and ys {list(ys.shape)} on {ys.device} do not belong together")
    k = _inv(fn, inv, T, dev)
    _gates(fn, gates, T, k, dev)
    if out is None:
        out = torch.empty((rows, H), dtype=ys.dtype, device=dev)
    elif out.shape != (rows, H) or out.dtype is not ys.dtype or out.device != dev:
        _bad(f"{fn}: out must be {ys.dtype} [{rows}, {H}] on {dev}")
    dgates = torch.empty((T, k), dtype=torch.float32, device=dev)
    check(lib().moe_combine_backward(dy.data_ptr(), _float(fn, "dy", dy), _ld(fn, "dy", dy), ys.data_ptr(),
                                     _float(fn, "ys", ys), _ld(fn, "ys", ys), rows, T, k, H, inv.data_ptr(),
                                     _ptr(gates), out.data_ptr(), _ld(fn, "out", out), dgates.data_ptr(),
                                     _raw_stream(dev.index)))
    return out, dgates
