"""GB300-native token layout, dispatch and combine of one MoE expert-parallel
(EP) layer whose R ranks are partitions of one GPU's HBM.

The product is the C-ABI library libep.so (include/ep.h, include/ep_ops.h),
built from the sm_103a CUDA sources in csrc/ by build.py.  This package holds
that build script, a ctypes binding with the ABI's names (_ep) and torch-facing
wrappers that allocate caller-owned outputs and pass device pointers and
streams: EpLayer (layer.py) and the operators around it (ops.py: the residual
norm to 8-bit rows, the router, the experts' products, the sum of a row's
picks).  Using EpLayer or _ep without a built libep.so raises ImportError:
there is no fallback path.  (The exports load lazily so that build.py can be
imported before the library exists.)
"""

_LAYER = ("EpLayer", "Layout", "ExpertLayout", "SmSplit", "CMD_DTYPE")
_OPS = ("Fp8Rows", "Normed", "Routing", "rms_norm", "rms_norm_backward", "route", "route_backward",
        "expert_product", "pick_sum")

__all__ = [*_LAYER, "EpError", *_OPS]


def __getattr__(name):
    if name in _LAYER:
        from . import layer as home
    elif name in _OPS:
        from . import ops as home
    elif name == "EpError":
        from . import _ep as home
    else:
        raise AttributeError(name)
    value = globals()[name] = getattr(home, name)      # found here from now on
    return value
