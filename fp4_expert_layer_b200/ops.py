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
their own: nothing here records an autograd graph.  So while grad mode is on an
``out`` that requires grad is refused, and an input that does (but for
``fp4_quantize``, whose codes have no gradient) is warned of; any ``out`` counts
as modified in place.
"""
from __future__ import annotations

import ctypes as C
from typing import NamedTuple, Optional

import torch

from ._lib import MoEError, lib

try:
    from . import _ops
except ImportError as e:
    raise ImportError("the operators' binding is not built (run fp4_expert_layer_b200/build.py)") from e
if _ops.built_for != torch.__version__:
    raise ImportError(f"the operators' binding was built for torch {_ops.built_for}, this is {torch.__version__}: "
                      "run fp4_expert_layer_b200/build.py")


class FP4Tensor(NamedTuple):
    """FP4 values in checkpoint layout: ``codes`` uint8 [..., K/2], ``scales`` uint8
    [..., K/32] (mxfp4) or [..., K/16] (nvfp4), ``global_scale`` fp32 (nvfp4, else
    None) with one value for each row, or for each matrix of a 3-D tensor."""
    codes: torch.Tensor
    scales: torch.Tensor
    global_scale: Optional[torch.Tensor]
    fmt: str


_ops.setup(MoEError, FP4Tensor, *(C.cast(getattr(lib(), "moe_" + n), C.c_void_p).value for n in (
    "fp4_quantize", "fp4_dequantize", "fp4_matmul", "sort_tokens", "dispatch", "dispatch_backward", "combine",
    "combine_backward", "last_error")))


def _elsewhere(fn, stream, *args):
    """fn(*args) with the first tensor's device current and, if given, on `stream`: what
    the call allocates belongs to that stream, and what it uses is kept for it."""
    t = args[0][0] if isinstance(args[0], tuple) and args[0] else args[0]
    if not isinstance(t, torch.Tensor):
        raise MoEError(1, f"{fn.__name__}: the first argument must hold tensors, not {type(t).__name__}")
    dev = t.device
    if dev.type != "cuda":
        raise MoEError(1, f"{fn.__name__}: the tensors must be CUDA tensors, not on {dev}")
    with torch.cuda.device(dev):
        if stream is None:
            return fn(*args)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, dev) if stream else torch.cuda.default_stream(dev)
        if getattr(stream, "device", None) != dev:
            raise MoEError(1, f"{fn.__name__}: the tensors are on {dev}, {stream} is no stream of it")
        with torch.cuda.stream(stream):
            got = fn(*args)
            for a in args:
                for t in a if isinstance(a, tuple) else (a,):
                    if isinstance(t, torch.Tensor):
                        t.record_stream(stream)
            return got


# The compiled functions check every argument, allocate, and call the library; they
# return None, having done nothing, when the tensors are not on the current device.

# ------------------------------------------------------------------------ FP4
def fp4_quantize(x, fmt="mxfp4", rows_per_scale=None, out=None, stream=None):
    """Quantise x [rows, K] or [matrices, rows, K] (float32, bfloat16, float16) to an
    :class:`FP4Tensor`.  nvfp4 has one fp32 scale for each ``rows_per_scale`` rows:
    by default one per row of a 2-D tensor, one per matrix of a 3-D one."""
    if stream is None:
        got = _ops.fp4_quantize(x, fmt, rows_per_scale, out)
        if got is not None:
            return got
    return _elsewhere(fp4_quantize, stream, x, fmt, rows_per_scale, out)


def fp4_dequantize(q, dtype=torch.float32, out=None, stream=None):
    """The values of an :class:`FP4Tensor`, each rounded once to ``dtype`` (float32 is
    exact with a global scale of at most 18 digits, as :func:`fp4_quantize` makes them,
    and within float32's range)."""
    if stream is None:
        got = _ops.fp4_dequantize(q, dtype, out)
        if got is not None:
            return got
    return _elsewhere(fp4_dequantize, stream, q, dtype, out)


def fp4_matmul(x, w, offsets=None, out_dtype=torch.bfloat16, out=None, stream=None):
    """x [rows, K] times the transpose of w [N, K] or, by groups of rows, of w [groups, N, K].

    Both are :class:`FP4Tensor` of one format (nvfp4: a global scale per row of x
    and per matrix of w).  ``offsets`` int32 [groups + 1] gives each group's rows
    (``sort_tokens`` writes it); without it w has one matrix and takes every row.
    Rows outside the groups are not written.  ``out`` takes the result in its own
    type.  Should a bounded wait of a product have given up on the GPU, that
    product's result is invalid, and the next call raises :class:`MoEError`, once
    (a call with no rows asks, and enqueues nothing)."""
    if stream is None:
        got = _ops.fp4_matmul(x, w, offsets, out_dtype, out)
        if got is not None:
            return got
    return _elsewhere(fp4_matmul, stream, x, w, offsets, out_dtype, out)


# ----------------------------------------------------------------- expert rows
def sort_tokens(ids, n_experts, stream=None):
    """Sort the pairs of ids int32 [T, k] by expert (stable).  Returns counts [E],
    offsets [E + 1], perm [T * k] (position -> pair, -1 behind the last) and inv
    [T, k] (pair -> position, -1 where the id is outside [0, E): a dropped pair)."""
    if stream is None:
        got = _ops.sort_tokens(ids, n_experts)
        if got is not None:
            return got
    return _elsewhere(sort_tokens, stream, ids, n_experts)


def dispatch(x, inv, rows=None, out=None, stream=None):
    """xs[inv[t, j]] = x[t].  x [T, H]: float32, bfloat16, float16 or uint8 (codes,
    scales); xs [rows, H], rows = T * k unless given (or out's); positions from
    ``rows`` on are dropped, rows that no pair names are not written."""
    if stream is None:
        got = _ops.dispatch(x, inv, rows, out)
        if got is not None:
            return got
    return _elsewhere(dispatch, stream, x, inv, rows, out)


def dispatch_backward(dxs, inv, out=None, stream=None):
    """Gradient of :func:`dispatch`: dx[t] = sum over t's pairs of dxs[inv[t, j]] (fp32, rounded once)."""
    if stream is None:
        got = _ops.dispatch_backward(dxs, inv, out)
        if got is not None:
            return got
    return _elsewhere(dispatch_backward, stream, dxs, inv, out)


def combine(ys, inv, gates=None, out_dtype=None, out=None, stream=None):
    """y[t] = sum over t's pairs of gates[t, j] * ys[inv[t, j]] (fp32, rounded once to
    ``out_dtype``, by default ys's).  gates fp32 [T, k], or None for ones."""
    if stream is None:
        got = _ops.combine(ys, inv, gates, out_dtype, out)
        if got is not None:
            return got
    return _elsewhere(combine, stream, ys, inv, gates, out_dtype, out)


def combine_backward(dy, ys, inv, gates=None, out=None, stream=None):
    """Gradients of :func:`combine`: (dys, dgates).  dys[inv[t, j]] = gates[t, j] * dy[t]
    in ys's type (``out`` takes it; rows that no pair names are not written);
    dgates[t, j] = <dy[t], ys[inv[t, j]]> fp32 [T, k], 0 for a dropped pair."""
    if stream is None:
        got = _ops.combine_backward(dy, ys, inv, gates, out)
        if got is not None:
            return got
    return _elsewhere(combine_backward, stream, dy, ys, inv, gates, out)
