"""ctypes binding of the sequence-mixing operators of ``libconvfwd.so`` (include/seq.h): a short
causal depthwise convolution, the selective state space scan it feeds, and the norm, gate and
residual step around such a block.

As in ``binding``, the functions carry the C-ABI names and only marshal arguments; the ``Seq...Plan``
classes check shapes and types, use PyTorch to allocate workspaces, and run every step in the
library's kernels.  Tensors lie on one token axis: ``(T, width)``, or ``(S, T/S, width)`` for
sequences of equal length; channels are contiguous, rows may be slices of a wider tensor.
"""
from __future__ import annotations

import ctypes
import struct

from .binding import CONV_BF16, CONV_ERR_INVALID_ARG, CONV_F32, CONV_OK, ConvError, load_library

__all__ = [
    "SEQ_FWD", "SEQ_BWD", "SEQ_STEP", "SEQ_RAGGED", "SEQ_CONV_SILU", "SEQ_SCAN_SOFTPLUS", "SEQ_NORM_LAYER_FLAG",
    "SEQ_NORM_POST", "SEQ_NORM_PRE", "SEQ_NORM_GATE_BEFORE", "SEQ_NORM_GATE_AFTER", "SEQ_NORM_RESIDUAL",
    "SEQ_NORM_RMS", "SEQ_NORM_LAYER", "SEQ_GATE_NONE", "SEQ_GATE_BEFORE", "SEQ_GATE_AFTER", "SEQ_EXPORTED",
    "seq_conv_plan_create", "seq_scan_plan_create", "seq_norm_plan_create", "seq_plan_describe",
    "seq_workspace_bytes", "seq_plan_set_workspace", "seq_plan_destroy", "seq_scan_saved_bytes",
    "SeqConvPlan", "SeqScanPlan", "SeqNormPlan",
]

SEQ_FWD, SEQ_BWD, SEQ_STEP = 0, 1, 2
SEQ_RAGGED, SEQ_CONV_SILU, SEQ_SCAN_SOFTPLUS, SEQ_NORM_LAYER_FLAG = 1, 2, 4, 8
SEQ_NORM_POST, SEQ_NORM_PRE, SEQ_NORM_GATE_BEFORE, SEQ_NORM_GATE_AFTER, SEQ_NORM_RESIDUAL = 16, 32, 64, 128, 256
SEQ_NORM_RMS, SEQ_NORM_LAYER = "rms", "layer"
SEQ_GATE_NONE, SEQ_GATE_BEFORE, SEQ_GATE_AFTER = "none", "before", "after"

_VP, _I64, _I, _U = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint
_PLAN = ctypes.POINTER(_VP)
_CALL = (ctypes.c_int, [_VP, ctypes.c_char_p, _VP])      # plan, argument struct, stream
_SIGS = {
    "seq_conv_plan_create": (ctypes.c_int, [_PLAN, _I64, _I64, _I64, _I64, _I, _I, _U]),
    "seq_scan_plan_create": (ctypes.c_int, [_PLAN, _I64, _I64, _I64, _I64, _I64, _I, _I, _U]),
    "seq_norm_plan_create": (ctypes.c_int, [_PLAN, _I64, _I64, _I, _I, _I, _U, ctypes.c_float]),
    "seq_plan_describe": (ctypes.c_char_p, [_VP]),
    "seq_workspace_bytes": (ctypes.c_size_t, [_VP]),
    "seq_plan_set_workspace": (ctypes.c_int, [_VP, _VP, ctypes.c_size_t]),
    "seq_plan_destroy": (ctypes.c_int, [_VP]),
    "seq_scan_saved_bytes": (ctypes.c_size_t, [_VP]),
    "seq_conv_fwd": _CALL, "seq_conv_bwd": _CALL, "seq_conv_step": _CALL,
    "seq_scan_fwd": _CALL, "seq_scan_bwd": _CALL, "seq_scan_step": _CALL,
    "seq_norm_fwd": _CALL, "seq_norm_bwd": _CALL,
}
SEQ_EXPORTED = tuple(_SIGS)
_bound = None

# The argument structs of include/seq.h as field names: every field is a pointer or an int64.
CONV_FIELDS = ("x", "x_ld", "w", "bias", "starts", "slots", "slot_count", "state_in", "state_out", "y", "y_ld",
               "dy", "dy_ld", "dx", "dx_ld", "dw", "dbias")
SCAN_FIELDS = ("x", "x_ld", "dt", "dt_ld", "A", "B", "B_ld", "C", "C_ld", "D", "z", "z_ld", "dt_bias", "starts",
               "slots", "slot_count", "h_in", "h_out", "y", "y_ld", "saved", "dy", "dy_ld", "dh_out", "dx", "dx_ld",
               "ddt", "ddt_ld", "dB", "dB_ld", "dC", "dC_ld", "dz", "dz_ld", "dA", "dD", "ddt_bias", "dh_in")
NORM_FIELDS = ("x", "x_ld", "gate", "gate_ld", "w_post", "b_post", "scale", "res", "res_ld", "w_pre", "b_pre", "y",
               "y_ld", "res_out", "res_out_ld", "dy", "dy_ld", "dres_out", "dres_out_ld", "dx", "dx_ld", "dgate",
               "dgate_ld", "dres", "dres_ld", "dw_post", "db_post", "dscale", "dw_pre", "db_pre")


def _bind(sigs):
    lib = load_library()
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


def _library():
    global _bound
    if _bound is None:
        _bound = _bind(_SIGS)
    return _bound


def _fail(what: str, why: str):
    raise ConvError(CONV_ERR_INVALID_ARG, f"{what}: {why}")


def _created(st, h, what):
    if st != CONV_OK:
        raise ConvError(st, what)
    return h.value


def seq_conv_plan_create(S, T, D, W, dtype, direction, flags) -> int:
    h = _VP()
    return _created(_library().seq_conv_plan_create(ctypes.byref(h), int(S), int(T), int(D), int(W), int(dtype),
                                                    int(direction), int(flags)), h, "seq_conv_plan_create")


def seq_scan_plan_create(S, T, D, N, G, dtype, direction, flags) -> int:
    h = _VP()
    return _created(_library().seq_scan_plan_create(ctypes.byref(h), int(S), int(T), int(D), int(N), int(G), int(dtype),
                                                    int(direction), int(flags)), h, "seq_scan_plan_create")


def seq_norm_plan_create(rows, D, dtype, res_dtype, direction, flags, eps) -> int:
    h = _VP()
    return _created(_library().seq_norm_plan_create(ctypes.byref(h), int(rows), int(D), int(dtype), int(res_dtype),
                                                    int(direction), int(flags), float(eps)), h, "seq_norm_plan_create")


def seq_plan_describe(plan: int) -> str:
    return _library().seq_plan_describe(plan).decode()


def seq_workspace_bytes(plan: int) -> int:
    return int(_library().seq_workspace_bytes(plan))


def seq_plan_set_workspace(plan: int, ptr: int, nbytes: int):
    st = _library().seq_plan_set_workspace(plan, ptr or None, int(nbytes))
    if st != CONV_OK:
        raise ConvError(st, "seq_plan_set_workspace")


def seq_scan_saved_bytes(plan: int) -> int:
    return int(_library().seq_scan_saved_bytes(plan))


def seq_plan_destroy(plan: int):
    st = _library().seq_plan_destroy(plan)
    if st != CONV_OK:
        raise ConvError(st, "seq_plan_destroy")


def _torch_dtype(code):
    import torch
    return torch.bfloat16 if code == CONV_BF16 else torch.float32


class _SeqPlan:
    """One plan and its workspace.  `direction` is "fwd", "bwd" or "step"; it decides which of
    `forward`, `backward` and `step` the plan runs."""

    _fields: tuple = ()
    _names: dict = {}

    def _open(self, handle, dtype, direction):
        import torch
        self.handle = handle
        self.dtype, self.direction = int(dtype), direction
        self.torch_dtype = _torch_dtype(dtype)
        self.workspace = None                    # of the latest call
        self._workspaces, self._ws_stream = {}, None      # stream -> its workspace; the stream of self.workspace
        self._f32, self._i32 = torch.float32, torch.int32
        self._ws_bytes = seq_workspace_bytes(handle)
        self._pack = struct.Struct(f"={len(self._fields)}q").pack
        self._place = {f: i for i, f in enumerate(self._fields)}
        self._blank = [0] * (len(self._fields) + 1)
        self._seen = {}          # argument -> the last layout found good for it
        self._state_shape = None                 # the same of the states
        name = self._names[direction]
        self._name, self._fn = name, getattr(_library(), name)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)      # (current_stream builds an object)
        self._stream = raw or (lambda index: torch.cuda.current_stream(index).cuda_stream)
        self._current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device

    @staticmethod
    def _direction(direction, allowed):
        if direction not in allowed:
            raise ValueError(f"unknown direction {direction!r}")
        return {"fwd": SEQ_FWD, "bwd": SEQ_BWD, "step": SEQ_STEP}[direction]

    def describe(self) -> str:
        return seq_plan_describe(self.handle)

    def allocate(self, device=None):
        """Allocate the workspace of the current stream, if the plan needs one (a call does so for its own stream)."""
        import torch
        if self._ws_bytes:
            index = device.index if isinstance(device, torch.device) else device
            index = torch.cuda.current_device() if index is None else index
            self._use_workspace(self._stream(index), index)
        return self

    def _use_workspace(self, s, index):
        """Take the workspace of stream s, allocated on that stream: PyTorch hands a freed block on in the order of
        the stream it was allocated on, so on another stream's block the kernels on s could meet the work of its last owner, or,
        once the plan is gone, of its next.  A plan keeps the workspaces of all its streams.  (A call that is being
        captured takes one that is there, since a graph runs on any stream: the plan must outlive the graph.)"""
        import torch
        ws = self._workspaces.get(s)
        if ws is None:
            on = torch.cuda.default_stream(index) if s == 0 else torch.cuda.ExternalStream(s, device=index)
            with torch.cuda.stream(on):
                if self._workspaces and torch.cuda.is_current_stream_capturing():
                    ws, s = next(iter(self._workspaces.values())), None
                else:
                    ws = torch.empty(self._ws_bytes, dtype=torch.uint8, device=torch.device("cuda", index))
                    self._workspaces[s] = ws
        self.workspace, self._ws_stream = ws, s
        seq_plan_set_workspace(self.handle, ws.data_ptr(), self._ws_bytes)

    # -- argument checks -------------------------------------------------------------------
    # `v` collects the values of the argument struct; behind them stands the device, x's, that all tensors are on.
    def _values(self, x, direction):
        if self.direction != direction:
            _fail(self._name, f"the plan's direction is {self.direction!r}")
        v = self._blank.copy()
        v[-1] = device = x.get_device()
        if device < 0 or device != self._current():
            _fail(self._name, f"x is on {x.device}, not on the current GPU")
        return v

    def _rows(self, v, name, t, width, dtype):
        """A tensor of the token axis: (rows, width), (1, rows, width) or (S, rows / S, width)."""
        if t is None:
            return
        sh, st = t.shape, t.stride()
        seen = self._seen.get(name)
        if seen is None or seen[0] != sh or seen[1] != st or seen[2] is not t.dtype or t.get_device() != v[-1]:
            seen = self._seen[name] = self._rows_layout(name, t, sh, st, width, dtype, v[-1])
        i = seen[4]
        v[i] = t.data_ptr()
        v[i + 1] = seen[3]

    def _rows_layout(self, name, t, sh, st, width, dtype, device):
        if t.dtype is not dtype or t.get_device() != device:
            _fail(self._name, f"{name} is not a {dtype} tensor on x's GPU")
        n = len(sh)
        if n == 2:
            rows, ld = sh[0], st[0]
        elif n == 3 and (sh[0] <= 1 or sh[1] <= 1 or st[0] == sh[1] * st[1]):
            rows, ld = sh[0] * sh[1], st[1]
            if sh[1] == 1:
                ld = st[0]
        else:
            _fail(self._name, f"{name} is not rows of one token axis: shape {tuple(sh)}, strides {tuple(st)}")
        if n == 3 and self._sequences and sh[0] > 1 and sh[1] > 1 and sh[0] != self._sequences:
            _fail(self._name, f"{name} has shape {tuple(sh)}: ({self._sequences}, {self._tokens // self._sequences}, {width}) or "
                              f"({self._tokens}, {width}) is wanted, sequences first")
        if rows != self._tokens or sh[-1] != width or (st[-1] != 1 and width > 1 and rows):
            _fail(self._name, f"{name} has shape {tuple(sh)}, strides {tuple(st)}: {self._tokens} rows of {width} contiguous "
                              "values are wanted")
        return sh, st, dtype, ld if rows > 1 else width, self._place[name]

    def _flat(self, v, name, t, shape, dtype):
        """A contiguous tensor of a fixed shape."""
        if t is None:
            return
        if t.dtype is not dtype or t.get_device() != v[-1] or t.shape != shape or not t.is_contiguous():
            _fail(self._name, f"{name} is not a contiguous {dtype} tensor of shape {tuple(shape)} on x's GPU")
        v[self._place[name]] = t.data_ptr()

    def _states(self, v, slots, starts, row, dtype, **states):
        """The state buffers: any number of rows of one shape; slots and starts."""
        count = -1
        for name, t in states.items():
            if t is None:
                continue
            sh = t.shape
            if (t.dtype is not dtype or t.get_device() != v[-1] or (sh != self._state_shape and sh[1:] != row)
                    or not t.is_contiguous()):
                _fail(self._name, f"{name} is not a contiguous {dtype} tensor of shape (slots, {', '.join(map(str, row))}) "
                                  "on x's GPU")
            if count >= 0 and sh[0] != count:
                _fail(self._name, "the state buffers have different numbers of rows")
            count = sh[0]
            self._state_shape = sh
            v[self._place[name]] = t.data_ptr()
        v[self._place["slot_count"]] = count if count > 0 else 0
        if slots is not None:
            self._flat(v, "slots", slots, (self.S,), self._i32)
        if starts is not None:
            self._flat(v, "starts", starts, (self.S + 1,), self._i32)

    def _call(self, v, device, stream):
        s = stream if stream is not None else self._stream(device)
        if self._ws_bytes and s != self._ws_stream:
            self._use_workspace(s, device)
        st = self._fn(self.handle, self._pack(*v), s)
        if st != CONV_OK:
            raise ConvError(st, self._name)

    def close(self):
        if getattr(self, "handle", 0):
            seq_plan_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class SeqConvPlan(_SeqPlan):
    """Short causal depthwise convolution of W taps over S sequences on T tokens of D channels
    (seq_conv_*).  w is (D, W), bias (D,); states are (slots, W - 1, D)."""

    _fields = CONV_FIELDS
    _names = {"fwd": "seq_conv_fwd", "bwd": "seq_conv_bwd", "step": "seq_conv_step"}

    def __init__(self, S, T, D, W, dtype, direction="fwd", ragged=False, silu=True):
        code = self._direction(direction, self._names)
        self.S, self.T, self.D, self.W = int(S), int(T), int(D), int(W)
        self._tokens, self._sequences = self.T, self.S
        self._width, self._taps, self._row = (self.D,), (self.D, self.W), (self.W - 1, self.D)
        self._open(seq_conv_plan_create(S, T, D, W, dtype, code, SEQ_RAGGED * bool(ragged) + SEQ_CONV_SILU * bool(silu)),
                   dtype, direction)

    def _common(self, direction, x, w, bias):
        v = self._values(x, direction)
        dt = self.torch_dtype
        self._rows(v, "x", x, self.D, dt)
        self._flat(v, "w", w, self._taps, dt)
        self._flat(v, "bias", bias, self._width, dt)
        return v

    def forward(self, x, w, bias, y, starts=None, state_in=None, state_out=None, slots=None, stream=None):
        v = self._common("fwd", x, w, bias)
        self._rows(v, "y", y, self.D, self.torch_dtype)
        self._states(v, slots, starts, self._row, self.torch_dtype, state_in=state_in, state_out=state_out)
        self._call(v, v.pop(), stream)
        return y

    def backward(self, x, w, bias, dy, dx, dw, dbias, starts=None, state_in=None, slots=None, stream=None):
        v = self._common("bwd", x, w, bias)
        self._rows(v, "dy", dy, self.D, self.torch_dtype)
        self._rows(v, "dx", dx, self.D, self.torch_dtype)
        self._flat(v, "dw", dw, (self.D, self.W), self._f32)
        self._flat(v, "dbias", dbias, (self.D,), self._f32)
        self._states(v, slots, starts, self._row, self.torch_dtype, state_in=state_in)
        self._call(v, v.pop(), stream)
        return dx, dw, dbias

    def step(self, x, w, bias, state_in, state_out, y, slots=None, stream=None):
        v = self._common("step", x, w, bias)
        self._rows(v, "y", y, self.D, self.torch_dtype)
        self._states(v, slots, None, self._row, self.torch_dtype, state_in=state_in, state_out=state_out)
        self._call(v, v.pop(), stream)
        return y


class SeqScanPlan(_SeqPlan):
    """Selective state space scan over S sequences on T tokens of D channels with N states each
    (seq_scan_*); B and C are shared by D / G channels.  A is (D, N), D and dt_bias are (D,), all
    float32; states are (slots, D, N) float32."""

    _fields = SCAN_FIELDS
    _names = {"fwd": "seq_scan_fwd", "bwd": "seq_scan_bwd", "step": "seq_scan_step"}

    def __init__(self, S, T, D, N, dtype, direction="fwd", G=1, ragged=False, softplus=True):
        code = self._direction(direction, self._names)
        self.S, self.T, self.D, self.N, self.G = int(S), int(T), int(D), int(N), int(G)
        self._tokens, self._sequences = self.T, self.S
        self._width, self._row = (self.D,), (self.D, self.N)
        self._open(seq_scan_plan_create(S, T, D, N, G, dtype, code,
                                        SEQ_RAGGED * bool(ragged) + SEQ_SCAN_SOFTPLUS * bool(softplus)), dtype, direction)
        self.saved_bytes = seq_scan_saved_bytes(self.handle)

    def allocate_saved(self, device=None):
        """A buffer for the states that `forward` saves for `backward`."""
        import torch
        return torch.empty(self.saved_bytes // 4, dtype=torch.float32,
                           device=device or torch.device("cuda", torch.cuda.current_device()))

    def _common(self, direction, x, dt, A, B, C, D, z, dt_bias):
        v = self._values(x, direction)
        td, f32 = self.torch_dtype, self._f32
        self._rows(v, "x", x, self.D, td)
        self._rows(v, "dt", dt, self.D, td)
        self._rows(v, "B", B, self.G * self.N, td)
        self._rows(v, "C", C, self.G * self.N, td)
        self._rows(v, "z", z, self.D, td)
        self._flat(v, "A", A, self._row, f32)
        self._flat(v, "D", D, self._width, f32)
        self._flat(v, "dt_bias", dt_bias, self._width, f32)
        return v

    def _saved(self, v, saved):
        if saved is not None:
            self._flat(v, "saved", saved, (self.saved_bytes // 4,), self._f32)

    def forward(self, x, dt, A, B, C, y, D=None, z=None, dt_bias=None, starts=None, h_in=None, h_out=None, slots=None,
                saved=None, stream=None):
        v = self._common("fwd", x, dt, A, B, C, D, z, dt_bias)
        self._rows(v, "y", y, self.D, self.torch_dtype)
        self._saved(v, saved)
        self._states(v, slots, starts, self._row, self._f32, h_in=h_in, h_out=h_out)
        self._call(v, v.pop(), stream)
        return y

    def backward(self, x, dt, A, B, C, dy, saved, dx, ddt, dA, dB, dC, D=None, z=None, dt_bias=None, dD=None, dz=None,
                 ddt_bias=None, starts=None, h_in=None, dh_out=None, dh_in=None, slots=None, stream=None):
        v = self._common("bwd", x, dt, A, B, C, D, z, dt_bias)
        td, f32 = self.torch_dtype, self._f32
        for name, t in (("dy", dy), ("dx", dx), ("ddt", ddt), ("dz", dz)):
            self._rows(v, name, t, self.D, td)
        self._rows(v, "dB", dB, self.G * self.N, td)
        self._rows(v, "dC", dC, self.G * self.N, td)
        self._flat(v, "dA", dA, (self.D, self.N), f32)
        self._flat(v, "dD", dD, (self.D,), f32)
        self._flat(v, "ddt_bias", ddt_bias, (self.D,), f32)
        self._saved(v, saved)
        self._states(v, slots, starts, self._row, f32, h_in=h_in, dh_out=dh_out, dh_in=dh_in)
        self._call(v, v.pop(), stream)
        return dx

    def step(self, x, dt, A, B, C, h_in, h_out, y, D=None, z=None, dt_bias=None, slots=None, stream=None):
        v = self._common("step", x, dt, A, B, C, D, z, dt_bias)
        self._rows(v, "y", y, self.D, self.torch_dtype)
        self._states(v, slots, None, self._row, self._f32, h_in=h_in, h_out=h_out)
        self._call(v, v.pop(), stream)
        return y


class SeqNormPlan(_SeqPlan):
    """Norm, gate and residual around a block on rows of D values (seq_norm_*): see include/seq.h
    for the formulas.  kind is SEQ_NORM_RMS or SEQ_NORM_LAYER, gate SEQ_GATE_NONE, SEQ_GATE_BEFORE or
    SEQ_GATE_AFTER (the POST norm).  The residual stream has the type res_dtype; `forward` may update it in place
    (res_out=res)."""

    _fields = NORM_FIELDS
    _names = {"fwd": "seq_norm_fwd", "bwd": "seq_norm_bwd"}

    def __init__(self, rows, D, dtype, direction="fwd", res_dtype=CONV_F32, kind=SEQ_NORM_RMS, post=False, pre=True,
                 gate=SEQ_GATE_NONE, residual=True, eps=1e-5):
        code = self._direction(direction, self._names)
        if kind not in (SEQ_NORM_RMS, SEQ_NORM_LAYER) or gate not in (SEQ_GATE_NONE, SEQ_GATE_BEFORE, SEQ_GATE_AFTER):
            raise ValueError(f"unknown kind {kind!r} or gate {gate!r}")
        flags = (SEQ_NORM_LAYER_FLAG * (kind == SEQ_NORM_LAYER) + SEQ_NORM_POST * bool(post) + SEQ_NORM_PRE * bool(pre) +
                 SEQ_NORM_GATE_BEFORE * (gate == SEQ_GATE_BEFORE) + SEQ_NORM_GATE_AFTER * (gate == SEQ_GATE_AFTER) +
                 SEQ_NORM_RESIDUAL * bool(residual))
        self.rows, self.D, self.eps = int(rows), int(D), float(eps)
        self._tokens, self._width = self.rows, (self.D,)
        self._sequences = None               # (rows have no order)
        self.res_torch_dtype = _torch_dtype(res_dtype)
        self._open(seq_norm_plan_create(rows, D, dtype, res_dtype, code, flags, eps), dtype, direction)

    def _common(self, direction, x, gate, w_post, b_post, scale, res, w_pre, b_pre):
        v = self._values(x, direction)
        td = self.torch_dtype
        self._rows(v, "x", x, self.D, td)
        self._rows(v, "gate", gate, self.D, td)
        self._rows(v, "res", res, self.D, self.res_torch_dtype)
        for name, t in (("w_post", w_post), ("b_post", b_post), ("scale", scale), ("w_pre", w_pre), ("b_pre", b_pre)):
            if t is not None:
                self._flat(v, name, t, self._width, td)
        return v

    def forward(self, x, y=None, gate=None, w_post=None, b_post=None, scale=None, res=None, res_out=None, w_pre=None,
                b_pre=None, stream=None):
        v = self._common("fwd", x, gate, w_post, b_post, scale, res, w_pre, b_pre)
        self._rows(v, "y", y, self.D, self.torch_dtype)
        self._rows(v, "res_out", res_out, self.D, self.res_torch_dtype)
        self._call(v, v.pop(), stream)
        return y, res_out

    def backward(self, x, dx, dy=None, dres_out=None, gate=None, w_post=None, b_post=None, scale=None, res=None,
                 w_pre=None, b_pre=None, dgate=None, dres=None, dw_post=None, db_post=None, dscale=None, dw_pre=None,
                 db_pre=None, stream=None):
        v = self._common("bwd", x, gate, w_post, b_post, scale, res, w_pre, b_pre)
        td, rd = self.torch_dtype, self.res_torch_dtype
        for name, t, dt in (("dy", dy, td), ("dres_out", dres_out, rd), ("dx", dx, td), ("dgate", dgate, td), ("dres", dres, rd)):
            self._rows(v, name, t, self.D, dt)
        for name, t in (("dw_post", dw_post), ("db_post", db_post), ("dscale", dscale), ("dw_pre", dw_pre),
                        ("db_pre", db_pre)):
            self._flat(v, name, t, (self.D,), self._f32)
        self._call(v, v.pop(), stream)
        return dx
