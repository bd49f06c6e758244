"""Host-side checks of the sequence-mixing operators that need no GPU: exported symbols, argument
structs, plan and call refusals, and the 64-bit oracle's gradients against differences.  No call
here launches a kernel."""
import ctypes
import os
import re

import numpy as np
import pytest

from convolution_forward_implicit_gb300 import binding as B
from convolution_forward_implicit_gb300 import seq as Q
from tests import seq_oracle as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "seq.h")).read(), flags=re.S)


@pytest.fixture(scope="module")
def lib():
    from convolution_forward_implicit_gb300.build import build_library
    build_library()
    return Q._library()


def test_library_exports_every_declared_symbol(lib):
    names = set(re.findall(r"^\s*(?:const\s+)?[a-z_][a-z_0-9]*\**\s+\**(seq_[a-z_0-9]+)\s*\(", HEADER, re.M))
    assert len(names) == 16
    for n in names:
        assert hasattr(lib, n), n
    assert names == set(Q.SEQ_EXPORTED)


@pytest.mark.parametrize("name,fields", [("conv", Q.CONV_FIELDS), ("scan", Q.SCAN_FIELDS), ("norm", Q.NORM_FIELDS)])
def test_argument_structs_match_the_header(name, fields):
    body = re.search(r"typedef struct \{([^}]*)\} seq_%s_args;" % name, HEADER, re.S).group(1)
    assert tuple(re.findall(r"(\w+);", body)) == fields


def _conv(S=2, T=8, D=16, W=4, dtype=B.CONV_BF16, direction=Q.SEQ_FWD, flags=Q.SEQ_CONV_SILU):
    return Q.seq_conv_plan_create(S, T, D, W, dtype, direction, flags)


def _scan(S=2, T=8, D=16, N=16, G=1, dtype=B.CONV_BF16, direction=Q.SEQ_FWD, flags=Q.SEQ_SCAN_SOFTPLUS):
    return Q.seq_scan_plan_create(S, T, D, N, G, dtype, direction, flags)


def _norm(rows=8, D=16, dtype=B.CONV_BF16, res=B.CONV_F32, direction=Q.SEQ_FWD,
          flags=Q.SEQ_NORM_PRE | Q.SEQ_NORM_RESIDUAL, eps=1e-5):
    return Q.seq_norm_plan_create(rows, D, dtype, res, direction, flags, eps)


@pytest.mark.parametrize("make,kw,status", [
    (_conv, dict(S=0), 1), (_conv, dict(T=-1), 1), (_conv, dict(D=0), 1), (_conv, dict(W=0), 1), (_conv, dict(W=9), 2),
    (_conv, dict(T=9), 1), (_conv, dict(dtype=5), 1), (_conv, dict(direction=3), 1), (_conv, dict(flags=4), 1),
    (_conv, dict(S=1, T=(1 << 30) + 1), 2), (_conv, dict(D=(1 << 22) + 1), 2),
    (_conv, dict(direction=Q.SEQ_STEP), 1), (_conv, dict(T=2, direction=Q.SEQ_STEP, flags=Q.SEQ_RAGGED), 1),
    (_scan, dict(N=0), 1), (_scan, dict(N=129), 2), (_scan, dict(G=3), 1), (_scan, dict(G=0), 1), (_scan, dict(T=7), 1),
    (_scan, dict(flags=2), 1), (_scan, dict(direction=Q.SEQ_STEP), 1), (_scan, dict(dtype=-1), 1),
    (_norm, dict(rows=0), 1), (_norm, dict(D=0), 1), (_norm, dict(D=16385), 2), (_norm, dict(flags=0), 1),
    (_norm, dict(flags=Q.SEQ_NORM_POST | Q.SEQ_NORM_GATE_BEFORE | Q.SEQ_NORM_GATE_AFTER), 1), (_norm, dict(eps=-1.0), 1),
    (_norm, dict(eps=float("nan")), 1), (_norm, dict(direction=Q.SEQ_STEP), 1), (_norm, dict(flags=Q.SEQ_NORM_PRE | 1), 1),
    (_norm, dict(dtype=B.CONV_F32, res=B.CONV_BF16), 2),
])
def test_plans_refuse_what_they_do_not_take(lib, make, kw, status):
    with pytest.raises(B.ConvError) as e:
        make(**kw)
    assert e.value.status == status


def _status(lib, name, plan, fields, **values):
    v = [int(values.pop(f, 0)) for f in fields]
    assert not values
    arr = (ctypes.c_int64 * len(v))(*v)
    return getattr(lib, name)(plan, ctypes.cast(arr, ctypes.c_char_p), None)


P = 1 << 20          # an address that is never read: every call below is refused before a launch


def test_conv_calls_check_their_arguments(lib):
    good = dict(x=P, x_ld=16, w=P, y=P, y_ld=16)
    st = lambda plan, name="seq_conv_fwd", **kw: _status(lib, name, plan, Q.CONV_FIELDS, **kw)      # noqa: E731
    fwd, bwd, rag = _conv(), _conv(direction=Q.SEQ_BWD), _conv(flags=Q.SEQ_RAGGED)
    assert st(None, **good) == 1 and st(bwd, **good) == 1 and st(fwd, "seq_conv_step", **good) == 1
    for k in ("x", "w", "y"):
        assert st(fwd, **{**good, k: 0}) == 1, k
        assert st(fwd, **{**good, k: P + 1}) == 3, k
    assert st(fwd, **{**good, "x_ld": 15}) == 1 and st(fwd, **{**good, "y_ld": 0}) == 1
    assert st(fwd, **good, starts=P) == 1 and st(rag, **good) == 1
    assert st(fwd, **good, state_in=P, slot_count=1) == 1          # fewer rows than sequences
    assert st(fwd, **good, state_in=P, slots=P, slot_count=-1) == 1
    b = dict(x=P, x_ld=16, w=P, dy=P, dy_ld=16, dx=P, dx_ld=16, dw=P)
    assert st(bwd, "seq_conv_bwd", **b) == 4                        # no workspace
    assert st(bwd, "seq_conv_bwd", **{**b, "dw": P + 2}) == 3
    assert st(bwd, "seq_conv_bwd", **b, dbias=P) == 1               # a gradient without its parameter
    one = _conv(W=1)
    assert st(one, **good, state_in=P, state_out=P, slot_count=2) == 1   # one tap keeps no state
    for p in (fwd, bwd, rag, one):
        Q.seq_plan_destroy(p)


def test_scan_calls_check_their_arguments(lib):
    good = dict(x=P, x_ld=16, dt=P, dt_ld=16, A=P, B=P, B_ld=16, C=P, C_ld=16, y=P, y_ld=16)
    st = lambda plan, name="seq_scan_fwd", **kw: _status(lib, name, plan, Q.SCAN_FIELDS, **kw)      # noqa: E731
    fwd, bwd = _scan(), _scan(direction=Q.SEQ_BWD)
    assert st(bwd, **good) == 1
    for k in ("x", "dt", "A", "B", "C", "y"):
        assert st(fwd, **{**good, k: 0}) == 1, k
        assert st(fwd, **{**good, k: P + 1}) == 3, k
    assert st(fwd, **{**good, "B_ld": 15}) == 1
    assert st(fwd, **good, z=P, z_ld=8) == 1
    assert st(fwd, **good, saved=P + 4) == 3
    assert st(fwd, **good, h_out=P, slot_count=1) == 1
    b = {**good, **dict(dy=P, dy_ld=16, dx=P, dx_ld=16, ddt=P, ddt_ld=16, dB=P, dB_ld=16, dC=P, dC_ld=16, dA=P, saved=P)}
    assert st(bwd, "seq_scan_bwd", **b) == 4
    for k in ("dy", "saved", "dx", "ddt", "dB", "dC", "dA"):
        assert st(bwd, "seq_scan_bwd", **{**b, k: 0}) == 1, k
    for k in ("dD", "ddt_bias"):
        assert st(bwd, "seq_scan_bwd", **b, **{k: P}) == 1, k
    assert st(bwd, "seq_scan_bwd", **b, D=P) == 1 and st(bwd, "seq_scan_bwd", **b, z=P, z_ld=16) == 1
    for p in (fwd, bwd):
        Q.seq_plan_destroy(p)


def test_norm_calls_check_their_arguments(lib):
    good = dict(x=P, x_ld=16, res=P, res_ld=16, res_out=P, res_out_ld=16, y=P, y_ld=16)
    st = lambda plan, name="seq_norm_fwd", **kw: _status(lib, name, plan, Q.NORM_FIELDS, **kw)      # noqa: E731
    fwd, bwd = _norm(), _norm(direction=Q.SEQ_BWD)
    for k in ("x", "res", "res_out", "y"):
        assert st(fwd, **{**good, k: 0}) == 1, k
        assert st(fwd, **{**good, k: P + 1}) == 3, k
    for k in ("gate", "w_post", "b_post"):                          # not part of this plan
        assert st(fwd, **good, **{k: P}, **({"gate_ld": 16} if k == "gate" else {})) == 1, k
    b = dict(x=P, x_ld=16, res=P, res_ld=16, dy=P, dy_ld=16, dx=P, dx_ld=16, dres=P, dres_ld=16)
    assert st(bwd, "seq_norm_bwd", **b, w_pre=P, dw_pre=P) == 4
    assert st(bwd, "seq_norm_bwd", **b, dw_pre=P) == 1
    for k in ("x", "res", "dy", "dx", "dres"):
        assert st(bwd, "seq_norm_bwd", **{**b, k: 0}) == 1, k
    for p in (fwd, bwd):
        Q.seq_plan_destroy(p)


def test_workspaces(lib):
    p = _conv(direction=Q.SEQ_BWD)
    need = Q.seq_workspace_bytes(p)
    assert need > 0 and lib.seq_plan_set_workspace(p, P, need - 1) == 4
    assert lib.seq_plan_set_workspace(p, P + 8, need) == 3 and lib.seq_plan_set_workspace(p, P, need) == 0
    Q.seq_plan_destroy(p)
    assert lib.seq_workspace_bytes(None) == 0 and lib.seq_scan_saved_bytes(None) == 0
    assert lib.seq_plan_set_workspace(None, P, 1) == 1 and lib.seq_plan_destroy(None) == 0
    f, b = _scan(T=50, D=12, N=6), _scan(T=50, D=12, N=6, direction=Q.SEQ_BWD)
    assert Q.seq_scan_saved_bytes(f) == Q.seq_scan_saved_bytes(b) > 0
    Q.seq_plan_destroy(f)
    Q.seq_plan_destroy(b)


def test_python_plans_refuse_tensors_that_do_not_fit(lib):
    import torch
    p = Q.SeqConvPlan(2, 8, 16, 4, B.CONV_F32)
    x, w = torch.zeros(8, 16), torch.zeros(16, 4)
    for bad in (x, torch.zeros(8, 16, dtype=torch.bfloat16), torch.zeros(7, 16)):       # not on the GPU, type, rows
        with pytest.raises(B.ConvError) as e:
            p.forward(bad, w, None, x)
        assert e.value.status == B.CONV_ERR_INVALID_ARG
    with pytest.raises(B.ConvError):
        p.backward(x, w, None, x, x, w, None)
    with pytest.raises(ValueError):
        Q.SeqConvPlan(2, 8, 16, 4, B.CONV_F32, direction="sideways")
    p.close()


# ------------------------------------------------------- the oracle's gradients against differences
def _directional(f, args, grads, name, rng, eps=1e-5):
    d = rng.standard_normal(args[name].shape)
    hi, lo = dict(args), dict(args)
    hi[name], lo[name] = args[name] + eps * d, args[name] - eps * d
    num = (f(**hi) - f(**lo)) / (2 * eps)
    ana = float((grads["d" + name] * d).sum())
    assert abs(num - ana) <= 1e-6 * max(1.0, abs(ana)), (name, num, ana)


def test_conv_gradients_against_differences():
    rng = np.random.default_rng(1)
    lens, D, W = [5, 0, 1, 7], 6, 4
    a = dict(x=rng.standard_normal((13, D)), w=rng.standard_normal((D, W)), bias=rng.standard_normal(D))
    state, dy = rng.standard_normal((4, W - 1, D)), rng.standard_normal((13, D))
    f = lambda x, w, bias: float((O.conv(x, w, bias, lens, state)[0] * dy).sum())       # noqa: E731
    g, _ = O.conv_grad(**a, lens=lens, state=state, dy=dy)
    for k in a:
        _directional(f, a, g, k, rng)


@pytest.mark.parametrize("act", [True, False])
def test_scan_gradients_against_differences(act):
    rng = np.random.default_rng(2)
    lens, W, N, G, T = [5, 0, 1, 7], 6, 3, 2, 13
    a = dict(x=rng.standard_normal((T, W)), dt=rng.standard_normal((T, W)) * 0.3 + (0 if act else 0.5),
             A=-rng.uniform(0.5, 2, (W, N)), B=rng.standard_normal((T, G * N)), C=rng.standard_normal((T, G * N)),
             D=rng.standard_normal(W), z=rng.standard_normal((T, W)), dt_bias=rng.standard_normal(W) * 0.2)
    h0, dy, dh = rng.standard_normal((4, W, N)), rng.standard_normal((T, W)), rng.standard_normal((4, W, N))

    def f(h_in=h0, **kw):
        o, _ = O.scan(**kw, G=G, lens=lens, h0=h_in, act=act)
        return float((o["y"] * dy).sum() + (o["h"] * dh).sum())

    g, _ = O.scan(**a, G=G, lens=lens, h0=h0, act=act, dy=dy, dh_out=dh)
    full = dict(a, h_in=h0)
    for k in full:
        _directional(f, full, g, k, rng)


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("post,pre,gate,after,res", [(1, 1, 1, 0, 1), (1, 1, 1, 1, 1), (0, 1, 0, 0, 1), (1, 0, 1, 1, 0),
                                                     (1, 0, 0, 0, 1), (0, 1, 1, 0, 0)])
def test_norm_gradients_against_differences(layer, post, pre, gate, after, res):
    rng = np.random.default_rng(3)
    R, D = 3, 7
    n = lambda *s: rng.standard_normal(s)       # noqa: E731
    a = dict(x=n(R, D), gate=n(R, D) if gate else None, w_post=n(D) if post else None, b_post=n(D) if post else None,
             scale=n(D), res=n(R, D) if res else None, w_pre=n(D) if pre else None, b_pre=n(D) if pre else None)
    dy, dres = n(R, D), n(R, D) if res else None

    def f(**kw):
        o, _ = O.norm(**kw, layer=layer, eps=1e-3, post=post, pre=pre, after=bool(after))
        return float((o["y"] * dy).sum() if "y" in o else 0) + float((o["res_out"] * dres).sum() if res else 0)

    g, _ = O.norm(**a, layer=layer, eps=1e-3, post=post, pre=pre, after=bool(after), dy=dy, dres_out=dres)
    for k in a:
        if a[k] is not None:
            _directional(f, a, g, k, rng)


# ------------------------------------------------------------------ the Python plans without a GPU
def test_a_workspace_is_allocated_on_the_stream_that_uses_it(lib, monkeypatch):
    """The allocator orders a block's owners by the stream it was allocated on.  Streams and memory are stood in
    for by numbers and host memory, the call by a function that notes the plan's workspace."""
    import contextlib
    import torch
    current, made, used = [7], [], []

    @contextlib.contextmanager
    def on(s):
        before, current[0] = current[0], s
        yield
        current[0] = before

    empty = torch.empty
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda s, device=None: s)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: 0)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: current[0] >= 100)
    p = Q.SeqConvPlan(2, 8, 16, 4, B.CONV_F32, direction="bwd")
    v = [0] * len(Q.CONV_FIELDS)
    p._stream = lambda index: current[0]
    p._fn = lambda handle, args, s: used.append((s, p.workspace.data_ptr())) or 0
    monkeypatch.setattr(torch, "empty", lambda n, dtype=None, device=None: made.append(current[0]) or empty(n, dtype=dtype))
    p._call(v, 0, 9)                 # a first call on another stream than the current one
    assert made == [9]
    p._call(v, 0, None)
    p._call(v, 0, 0)
    assert made == [9, 7, 0]
    for s in (9, None, 0, 9):        # every stream keeps its own
        p._call(v, 0, s)
    assert made == [9, 7, 0] and current == [7]
    at = dict(used)
    assert len(set(at.values())) == 3 and all(at[s] == w for s, w in used)
    p._call(v, 0, 100)               # captured: one that is there, and nothing allocated
    assert made == [9, 7, 0] and used[-1][1] in at.values()
    p._call(v, 0, None)
    assert used[-1] == (7, at[7])
    p.close()
    q = Q.SeqConvPlan(2, 8, 16, 4, B.CONV_F32, direction="bwd")
    q._stream = p._stream
    q.allocate(torch.device("cuda", 0)).allocate(0)
    assert made == [9, 7, 0, 7]
    q.close()


class OnGpu:
    """What the plans' layout checks look at in a tensor, of a tensor that is not there."""
    is_cuda = True

    def __init__(self, host):
        self.dtype, self.shape, self.stride = host.dtype, host.shape, host.stride

    def data_ptr(self):
        return P

    def get_device(self):
        return 0


def _layout(plan, host, width):
    v = [0] * len(plan._fields)
    plan._rows(v, "x", OnGpu(host), width, plan.torch_dtype)
    assert v[plan._place["x"]] == P
    return v[plan._place["x_ld"]]


@pytest.mark.parametrize("make", [lambda **k: Q.SeqConvPlan(4, 24, 16, 4, B.CONV_F32, **k), lambda **k: Q.SeqScanPlan(4, 24, 16, 8, B.CONV_F32, **k)])
def test_python_plans_take_sequences_first(lib, make):
    """(L, S, D) has as many rows as (S, L, D), in another order."""
    import torch
    for p in (make(), make(ragged=True)):
        for good, ld in ((torch.zeros(24, 16), 16), (torch.zeros(24, 20)[:, 4:], 20), (torch.zeros(4, 6, 16), 16), (torch.zeros(1, 24, 16), 16),
                         (torch.zeros(4, 6, 40)[..., :16], 40), (torch.zeros(24, 1, 16), 16)):
            assert _layout(p, good, 16) == ld
        for bad in (torch.zeros(6, 4, 16), torch.zeros(2, 12, 16), torch.zeros(6, 4, 16).transpose(0, 1)):
            with pytest.raises(B.ConvError) as e:
                _layout(p, bad, 16)
            assert e.value.status == B.CONV_ERR_INVALID_ARG
        p.close()
    n = Q.SeqNormPlan(24, 16, B.CONV_F32)             # its rows have no order
    assert _layout(n, torch.zeros(6, 4, 16), 16) == 16 and _layout(n, torch.zeros(4, 6, 16), 16) == 16
    n.close()


def test_python_plans_take_one_token_of_longer_sequences(lib):
    """x[:, -1:, :] of (S, L, D): rows that lie L tokens apart."""
    import torch
    x = torch.zeros(4, 6, 20)
    for p in (Q.SeqConvPlan(4, 4, 16, 4, B.CONV_F32, direction="step"), Q.SeqScanPlan(4, 4, 16, 8, B.CONV_F32, direction="step"),
              Q.SeqNormPlan(4, 16, B.CONV_F32)):
        assert _layout(p, x[:, 5, :16], 16) == 120 and _layout(p, x[:, 5:, :16], 16) == 120
        p.close()
    p = Q.SeqConvPlan(1, 1, 16, 4, B.CONV_F32, direction="step")
    assert _layout(p, x[:1, 5:, :16], 16) == 16          # one row: its distance to the next does not matter
    p.close()


class On(OnGpu):
    """The same on a certain GPU, with the strides of `host` and any device."""

    def __init__(self, host, device=0):
        super().__init__(host)
        self.at, self.is_contiguous, self.device = device, host.is_contiguous, f"cuda:{device}"

    def get_device(self):
        return self.at


@pytest.mark.parametrize("current", [0, 1])
def test_python_plans_want_every_tensor_on_the_launching_gpu(lib, current):
    import torch
    z = torch.zeros
    calls = []

    def ready(p):
        p._current, p._stream, p._fn = (lambda: current), (lambda index: 0), (lambda *a: calls.append(a) or 0)
        return p

    conv = ready(Q.SeqConvPlan(2, 8, 16, 4, B.CONV_F32))
    scan = ready(Q.SeqScanPlan(2, 8, 16, 8, B.CONV_F32, ragged=True))
    norm = ready(Q.SeqNormPlan(8, 16, B.CONV_F32))
    a = dict(x=z(8, 16), w=z(16, 4), bias=z(16), y=z(8, 16), state_in=z(2, 3, 16), slots=z(2, dtype=torch.int32))
    b = dict(x=z(8, 16), dt=z(8, 16), A=z(16, 8), B=z(8, 8), C=z(8, 8), y=z(8, 16), D=z(16), h_in=z(2, 16, 8), starts=z(3, dtype=torch.int32))
    c = dict(x=z(8, 16), y=z(8, 16), res=z(8, 16), res_out=z(8, 16), w_pre=z(16))
    for plan, args in ((conv, a), (scan, b), (norm, c)):
        on = {k: On(t, current) for k, t in args.items()}
        n = len(calls)
        plan.forward(**on)
        assert len(calls) == n + 1
        for k, t in args.items():                 # one of them elsewhere, after the same call was good
            with pytest.raises(B.ConvError) as e:
                plan.forward(**{**on, k: On(t, 1 - current)})
            assert e.value.status == B.CONV_ERR_INVALID_ARG
        with pytest.raises(B.ConvError):          # all of them on a GPU that is not the current one
            plan.forward(**{k: On(t, 1 - current) for k, t in args.items()})
        assert len(calls) == n + 1
        plan.close()


def test_arguments_read_by_elements_do_not_choose_the_kernel(tmp_path):
    """Rows in aligned groups have kernels of their own.  Only what those read or write in groups decides; bounds,
    slots, single parameters, the scan's B and C and parameter gradients may lie at any element."""
    import shutil
    import subprocess
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists(os.path.join(cuda, "cuda.h")):
        pytest.skip("needs g++ and the CUDA headers")
    exe = tmp_path / "seq_dispatch_check"
    subprocess.check_call([gxx, "-O1", "-std=c++17", "-I", os.path.join(ROOT, "convolution_forward_implicit_gb300", "csrc"), "-I",
                           os.path.join(ROOT, "include"), "-I", cuda, os.path.join(ROOT, "tests", "native", "seq_dispatch_check.cpp"), "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0, out.stdout + out.stderr
    got = {name: rest.split() for name, rest in (line.split(":") for line in out.stdout.splitlines())}
    both = lambda *names: [v for n in names for v in (n, n + "_ld")]      # noqa: E731
    params = ["w_post", "b_post", "scale", "w_pre", "b_pre"]
    assert got.pop("conv_fwd 1") == both("x") + ["state_in", "state_out"] + both("y")
    assert got.pop("conv_bwd 1") == both("x") + ["state_in"] + both("dy", "dx")
    assert got.pop("conv_step 1") == both("x") + ["state_in", "state_out"] + both("y")
    assert got.pop("scan_fwd 16") == both("x", "dt", "z", "y") and got.pop("scan_fwd quads 1") == ["A"]
    assert got.pop("scan_bwd 16") == both("x", "dt", "z", "dy", "dx", "ddt", "dz") and got.pop("scan_bwd quads 1") == ["A"]
    assert got.pop("scan_step 16") == both("x", "dt", "z", "y")
    assert got.pop("scan_step quads 1") == ["A"] + both("B", "C") + ["h_in", "h_out"]
    # (an fp32 residual's rows one element further are aligned to 4 bytes only)
    assert sorted(got.pop("norm_fwd 1")) == sorted(both("x", "gate", "res", "y", "res_out") + params)
    assert sorted(got.pop("norm_bwd 1")) == sorted(both("x", "gate", "res", "dy", "dres_out", "dx", "dgate", "dres") + params)
    assert not got, got


# ------------------------------------------------------ what the cases of long memory can tell
SLOW = [([1300], False), ([300, 1200], True), ([4100], False), ([1, 900, 0, 2100, 33, 777, 8, 450], True)]


@pytest.mark.parametrize("lens,ragged", SLOW)
def test_cases_of_long_memory_tell_wrong_joins(lens, ragged):
    """Joining the pieces of the token axis, with a mistake planted in it, leaves the bound that the kernels are held to
    in these cases."""
    rng = np.random.default_rng(len(lens))
    D, N = 12, 4
    a, more = O.slow_case(rng, lens, D, N)
    want, mag = O.scan(**a, G=1, lens=lens, h0=more["h"])
    k = 4 * max(lens) + N + 100
    piece, parts = (32, 4) if sum(lens) < 2048 else (40, 8)
    assert (parts == 4) == (sum(lens) <= 64 * piece)
    y, h = O.scan_in_pieces(**a, lens=lens, h0=more["h"], piece=piece, parts=parts)
    O.check("y", y, want["y"], mag["y"], k, True)
    O.check("h", h, want["h"], mag["h"], k, False)
    faults = ["parts before", "decay over a part"] + ["older parts"] * (len(lens) == 1) + ["ends of sequences"] * ragged
    for fault in faults:
        y, h = O.scan_in_pieces(**a, lens=lens, h0=more["h"], piece=piece, parts=parts, fault=fault)
        with pytest.raises(AssertionError):
            O.check("y", y, want["y"], mag["y"], k, True)
        with pytest.raises(AssertionError):
            O.check("h", h, want["h"], mag["h"], k, False)


def test_bounds_outside_their_contract_stay_inside_the_tensors(tmp_path):
    """include/seq.h: sequence bounds and slots outside their contract lead to no access outside the tensors.  The
    kernels' own lookups, compiled for the host, on such values."""
    import shutil
    import subprocess
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("needs g++")
    src = os.path.join(ROOT, "convolution_forward_implicit_gb300", "csrc")

    def cut(name, what):
        text = open(os.path.join(src, name)).read()
        i = text.index(what)
        j = text.index("\n};" if what.startswith("struct") else "\n}", i)
        return text[i:j] + ("\n};\n" if what.startswith("struct") else "\n}\n")

    d = "__device__ __forceinline__ "
    parts = [("seq_internal.h", d + "int seq_start("), ("seq_internal.h", d + "int seq_first_at("), ("seq_internal.h", d + "long long seq_slot("),
             ("seq_conv.cu", "struct Place {"), ("seq_conv.cu", d + "Place place_of("), ("seq_conv.cu", d + "void next_place("),
             ("seq_scan.cuh", "struct ScanPlace {"), ("seq_scan.cuh", d + "ScanPlace scan_place(")]
    (tmp_path / "seq_bounds.inc").write_text("".join(cut(*p) for p in parts))
    exe = tmp_path / "seq_bounds_check"
    subprocess.check_call([gxx, "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", str(tmp_path),
                           os.path.join(ROOT, "tests", "native", "seq_bounds_check.cpp"), "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and " 0 wrong" in out.stdout, out.stdout + out.stderr
