"""ctypes binding of the gated delta rule of ``libconvfwd.so`` (include/delta.h): a linear recurrence with
a matrix state for each value head, on the token axis of ``seq``.

As there, the functions carry the C-ABI names and only marshal arguments; ``SeqDeltaPlan`` checks shapes
and types, uses PyTorch to allocate workspaces, and runs every step in the library's kernels.  Tensors of
tokens are ``(T, width)``, or ``(S, T/S, width)`` for sequences of equal length; rows may be slices of a
wider tensor.
"""
from __future__ import annotations

import ctypes

from . import seq as _seq
from .binding import CONV_OK, ConvError
from .seq import SEQ_RAGGED, _SeqPlan

__all__ = ["SEQ_DELTA_QK_NORM", "DELTA_EXPORTED", "seq_delta_plan_create", "seq_delta_saved_bytes", "seq_delta_check",
           "SeqDeltaPlan"]

SEQ_DELTA_QK_NORM = 512

_I64, _I, _U = ctypes.c_int64, ctypes.c_int, ctypes.c_uint
_SIGS = {
    "seq_delta_plan_create": (ctypes.c_int, [_seq._PLAN, _I64, _I64, _I64, _I64, _I64, _I64, _I, _I, _U, ctypes.c_float]),
    "seq_delta_saved_bytes": (ctypes.c_size_t, [ctypes.c_void_p]),
    "seq_delta_check": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "seq_delta_fwd": _seq._CALL, "seq_delta_bwd": _seq._CALL, "seq_delta_step": _seq._CALL,
}
DELTA_EXPORTED = tuple(_SIGS)
_bound = None

# The argument struct of include/delta.h as field names: every field is a pointer or an int64.
DELTA_FIELDS = ("q", "q_ld", "k", "k_ld", "v", "v_ld", "g", "g_ld", "beta", "beta_ld", "starts", "slots", "slot_count",
                "h_in", "h_out", "y", "y_ld", "saved", "dy", "dy_ld", "dh_out", "dq", "dq_ld", "dk", "dk_ld", "dv", "dv_ld",
                "dg", "dg_ld", "dbeta", "dbeta_ld", "dh_in")


def _library():
    global _bound
    if _bound is None:
        _bound = _seq._bind(_SIGS)
    return _bound


def seq_delta_plan_create(S, T, Hk, Hv, Dk, Dv, dtype, direction, flags, scale=0.0) -> int:
    h = ctypes.c_void_p()
    return _seq._created(_library().seq_delta_plan_create(ctypes.byref(h), int(S), int(T), int(Hk), int(Hv), int(Dk), int(Dv),
                                                          int(dtype), int(direction), int(flags), float(scale)), h,
                         "seq_delta_plan_create")


def seq_delta_saved_bytes(plan: int) -> int:
    return int(_library().seq_delta_saved_bytes(plan))


def seq_delta_check(plan: int, stream: int):
    st = _library().seq_delta_check(plan, stream)
    if st != CONV_OK:
        raise ConvError(st, "seq_delta_check")


class SeqDeltaPlan(_SeqPlan):
    """Gated delta rule over S sequences on T tokens (seq_delta_*): Hk key heads of Dk values hold q and k, Hv value
    heads of Dv values v and y; g and beta are (T, Hv) float32, states (slots, Hv, Dk, Dv) float32.  `qk_norm` divides q
    and k of a head by their length; `scale` of y is 1 / sqrt(Dk) unless given."""

    _fields = DELTA_FIELDS
    _names = {"fwd": "seq_delta_fwd", "bwd": "seq_delta_bwd", "step": "seq_delta_step"}

    def __init__(self, S, T, Hk, Hv, Dk, Dv, dtype, direction="fwd", ragged=False, qk_norm=True, scale=None):
        code = self._direction(direction, self._names)
        self.S, self.T, self.Hk, self.Hv, self.Dk, self.Dv = int(S), int(T), int(Hk), int(Hv), int(Dk), int(Dv)
        if scale is not None and not ctypes.c_float(scale).value:       # (zero stands for 1 / sqrt(Dk) there)
            raise ValueError("scale is zero in fp32")
        self._tokens, self._sequences = self.T, self.S
        self._keys, self._values_width, self._row = self.Hk * self.Dk, self.Hv * self.Dv, (self.Hv, self.Dk, self.Dv)
        self._open(seq_delta_plan_create(S, T, Hk, Hv, Dk, Dv, dtype, code,
                                         SEQ_RAGGED * bool(ragged) + SEQ_DELTA_QK_NORM * bool(qk_norm), scale or 0.0),
                   dtype, direction)
        self.saved_bytes = seq_delta_saved_bytes(self.handle)

    def allocate_saved(self, device=None):
        """A buffer for what `forward` saves for `backward`."""
        import torch
        return torch.empty(self.saved_bytes // 4, dtype=torch.float32,
                           device=device or torch.device("cuda", torch.cuda.current_device()))

    def check(self, stream=None):
        """Wait for the stream; raise if a kernel's wait for the tensor cores ran out (see seq_delta_check)."""
        import torch
        seq_delta_check(self.handle, torch.cuda.current_stream().cuda_stream if stream is None else stream)

    def _common(self, direction, q, k, v, g, beta):
        vals = self._values(q, direction)
        td, f32 = self.torch_dtype, self._f32
        self._rows(vals, "q", q, self._keys, td)
        self._rows(vals, "k", k, self._keys, td)
        self._rows(vals, "v", v, self._values_width, td)
        self._rows(vals, "g", g, self.Hv, f32)
        self._rows(vals, "beta", beta, self.Hv, f32)
        return vals

    def _saved(self, vals, saved):
        if saved is not None:
            self._flat(vals, "saved", saved, (self.saved_bytes // 4,), self._f32)

    def forward(self, q, k, v, g, beta, y, starts=None, h_in=None, h_out=None, slots=None, saved=None, stream=None):
        vals = self._common("fwd", q, k, v, g, beta)
        self._rows(vals, "y", y, self._values_width, self.torch_dtype)
        self._saved(vals, saved)
        self._states(vals, slots, starts, self._row, self._f32, h_in=h_in, h_out=h_out)
        self._call(vals, vals.pop(), stream)
        return y

    def backward(self, q, k, v, g, beta, dy, saved, dq, dk, dv, dg, dbeta, starts=None, dh_out=None, dh_in=None, slots=None,
                 stream=None):
        vals = self._common("bwd", q, k, v, g, beta)
        td, f32 = self.torch_dtype, self._f32
        self._rows(vals, "dy", dy, self._values_width, td)
        self._rows(vals, "dq", dq, self._keys, td)
        self._rows(vals, "dk", dk, self._keys, td)
        self._rows(vals, "dv", dv, self._values_width, td)
        self._rows(vals, "dg", dg, self.Hv, f32)
        self._rows(vals, "dbeta", dbeta, self.Hv, f32)
        self._saved(vals, saved)
        self._states(vals, slots, starts, self._row, f32, dh_out=dh_out, dh_in=dh_in)
        self._call(vals, vals.pop(), stream)
        return dq, dk, dv

    def step(self, q, k, v, g, beta, h_in, h_out, y, slots=None, stream=None):
        vals = self._common("step", q, k, v, g, beta)
        self._rows(vals, "y", y, self._values_width, self.torch_dtype)
        self._states(vals, slots, None, self._row, self._f32, h_in=h_in, h_out=h_out)
        self._call(vals, vals.pop(), stream)
        return y
