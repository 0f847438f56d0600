"""One data-parallel rank's partitioned mixed-precision optimizer step (ZeRO
stage 1/2) on AMD Instinct MI355X: a thin binding of libzero_shard.so.

The C ABI's calls and structs are available here under their C names
(zero_shard_init, zero_reduce_grads, ...); ZeroShard, ZeroOffload and ZeroGrads
hold the caller-owned buffers of one handle and call them, ZeroPacked those of
one matrix in packed rows."""
from . import _abi
from ._abi import (ZERO_ACCUMULATED, ZERO_ACT_GELU, ZERO_ACT_SILU, ZERO_BF16, ZERO_CLIP_EACH, ZERO_CLIP_GLOBAL,
                   ZERO_DEVICE_LOSS_SCALE, ZERO_F16, ZERO_F32, ZERO_NORM_L2, ZERO_NORM_MAX, ZERO_PACKED_INPUT_GRAD,
                   ZERO_PACKED_LINEAR, ZERO_PACKED_WEIGHT_GRAD, ZERO_SCALE_MAX, ZERO_SCALE_POW2, ZeroError)

_C_NAMES = sorted(n for n in vars(_abi) if n.startswith("zero_"))
globals().update({n: getattr(_abi, n) for n in _C_NAMES})

__all__ = ["ZERO_F16", "ZERO_BF16", "ZERO_F32", "ZERO_ACCUMULATED", "ZERO_DEVICE_LOSS_SCALE", "ZERO_NORM_L2",
           "ZERO_NORM_MAX", "ZERO_CLIP_GLOBAL", "ZERO_CLIP_EACH", "ZERO_SCALE_POW2", "ZERO_SCALE_MAX", "ZERO_ACT_GELU",
           "ZERO_ACT_SILU", "ZERO_PACKED_LINEAR", "ZERO_PACKED_WEIGHT_GRAD", "ZERO_PACKED_INPUT_GRAD", "ZeroError",
           "ZeroShard", "ZeroOffload", "ZeroGrads", "ZeroPacked"] + _C_NAMES


def __getattr__(name):
    if name == "ZeroShard":
        from .shard import ZeroShard
        return ZeroShard
    if name == "ZeroOffload":
        from .offload import ZeroOffload
        return ZeroOffload
    if name == "ZeroGrads":
        from .grads import ZeroGrads
        return ZeroGrads
    if name == "ZeroPacked":
        from .packed import ZeroPacked
        return ZeroPacked
    raise AttributeError(name)
