"""ctypes binding of the group norm with an activation of ``libconvfwd.so`` (include/gnorm.h), channels last:
what stands between two convolutions.

As in ``seq``, the functions carry the C-ABI names and only marshal arguments; ``SeqGroupNormPlan`` checks shapes
and types, uses PyTorch to allocate workspaces, and runs every step in the library's kernels.  The output of a
convolution over N samples of L positions is S = N sequences on T = N L tokens: ``(N L, C)`` or ``(N, L, C)``.
"""
from __future__ import annotations

import ctypes

from . import seq as _seq
from .seq import SEQ_RAGGED, _SeqPlan

__all__ = ["SEQ_ACT_NONE", "SEQ_ACT_SILU", "SEQ_ACT_GELU", "GNORM_EXPORTED", "seq_gnorm_plan_create", "SeqGroupNormPlan"]

SEQ_ACT_NONE, SEQ_ACT_SILU, SEQ_ACT_GELU = 0, 1, 2
_ACTS = {"none": SEQ_ACT_NONE, "silu": SEQ_ACT_SILU, "gelu": SEQ_ACT_GELU}

_I64, _I, _U = ctypes.c_int64, ctypes.c_int, ctypes.c_uint
_SIGS = {
    "seq_gnorm_plan_create": (ctypes.c_int, [_seq._PLAN, _I64, _I64, _I64, _I64, _I, _I, _U, _I, ctypes.c_float]),
    "seq_gnorm_fwd": _seq._CALL, "seq_gnorm_bwd": _seq._CALL,
}
GNORM_EXPORTED = tuple(_SIGS)
_bound = None

# The argument struct of include/gnorm.h as field names: every field is a pointer or an int64.
GNORM_FIELDS = ("x", "x_ld", "w", "b", "starts", "stats", "y", "y_ld", "dy", "dy_ld", "dx", "dx_ld", "dw", "db")


def _library():
    global _bound
    if _bound is None:
        _bound = _seq._bind(_SIGS)
    return _bound


def seq_gnorm_plan_create(S, T, D, G, dtype, direction, flags, act, eps) -> int:
    h = ctypes.c_void_p()
    return _seq._created(_library().seq_gnorm_plan_create(ctypes.byref(h), int(S), int(T), int(D), int(G), int(dtype),
                                                          int(direction), int(flags), int(act), float(eps)), h,
                         "seq_gnorm_plan_create")


class SeqGroupNormPlan(_SeqPlan):
    """Group norm and activation over S sequences on T tokens of D channels in G groups (seq_gnorm_*).  act is "none",
    "silu" or "gelu"; w and b are (D,) or None; stats, (S, G, 2) float32, holds each group's mean and 1 / standard
    deviation: `forward` leaves them there if it is given, `backward` needs them."""

    _fields = GNORM_FIELDS
    _names = {"fwd": "seq_gnorm_fwd", "bwd": "seq_gnorm_bwd"}

    def __init__(self, S, T, D, G, dtype, direction="fwd", ragged=False, act="none", eps=1e-5):
        code = self._direction(direction, self._names)
        if act not in _ACTS:
            raise ValueError(f"unknown activation {act!r}")
        self.S, self.T, self.D, self.G, self.eps = int(S), int(T), int(D), int(G), float(eps)
        self._tokens, self._sequences = self.T, self.S
        self._width, self._stats, self._bounds = (self.D,), (self.S, self.G, 2), (self.S + 1,)
        self._open(seq_gnorm_plan_create(S, T, D, G, dtype, code, SEQ_RAGGED * bool(ragged), _ACTS[act], eps), dtype, direction)

    def _common(self, direction, x, w, b, starts, stats):
        v = self._values(x, direction)
        td = self.torch_dtype
        self._rows(v, "x", x, self.D, td)
        self._flat(v, "w", w, self._width, td)
        self._flat(v, "b", b, self._width, td)
        self._flat(v, "starts", starts, self._bounds, self._i32)
        self._flat(v, "stats", stats, self._stats, self._f32)
        return v

    def forward(self, x, y, w=None, b=None, starts=None, stats=None, stream=None):
        v = self._common("fwd", x, w, b, starts, stats)
        self._rows(v, "y", y, self.D, self.torch_dtype)
        self._call(v, v.pop(), stream)
        return y

    def backward(self, x, stats, dy, dx, w=None, b=None, dw=None, db=None, starts=None, stream=None):
        v = self._common("bwd", x, w, b, starts, stats)
        self._rows(v, "dy", dy, self.D, self.torch_dtype)
        self._rows(v, "dx", dx, self.D, self.torch_dtype)
        self._flat(v, "dw", dw, self._width, self._f32)
        self._flat(v, "db", db, self._width, self._f32)
        self._call(v, v.pop(), stream)
        return dx
