"""B200 (sm_100a) sparse MoE layer over MXFP4 / NVFP4 experts with a resident-slot table.

The compute path is the CUDA library ``libfp4moe.so`` (C ABI in
``include/moe_layer.h`` and, for the expert path's operators on their own,
``include/moe_ops.h``); this package is its Python binding.  Importing the
package does not load the library; creating a layer does, and fails loudly if
the library is missing.
"""
from ._lib import (MoEError, MoELayer, admit, lib, make_config, plan,  # noqa: F401
                   weights_from_layer)

__all__ = ["MoELayer", "MoEError", "make_config", "plan", "admit", "weights_from_layer", "lib"]

_OPS = ("FP4Tensor", "fp4_quantize", "fp4_dequantize", "fp4_matmul", "sort_tokens", "dispatch", "dispatch_backward",
        "combine", "combine_backward")
__all__ += _OPS


def __getattr__(name):
    # the operators take torch tensors: torch is imported with the first of them
    if name in _OPS:
        from . import ops
        globals().update({n: getattr(ops, n) for n in _OPS})
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
