"""Host-side checks of the gated delta rule and the group norm that need no GPU: exported symbols, argument structs, plan and
call refusals, and the 64-bit oracle's gradients against differences.  No call here launches a kernel."""
import ctypes
import os
import re

import numpy as np
import pytest

from convolution_forward_implicit_gb300 import binding as B
from convolution_forward_implicit_gb300 import delta as D
from convolution_forward_implicit_gb300 import gnorm as N
from convolution_forward_implicit_gb300 import seq as Q
from tests import delta_oracle as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def header(name):
    return re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", name)).read(), flags=re.S)


@pytest.fixture(scope="module")
def lib():
    from convolution_forward_implicit_gb300.build import build_library
    build_library()
    D._library()
    N._library()
    return Q._library()


@pytest.mark.parametrize("file,names,fields", [("delta.h", D.DELTA_EXPORTED, D.DELTA_FIELDS), ("gnorm.h", N.GNORM_EXPORTED, N.GNORM_FIELDS)])
def test_symbols_and_structs_match_the_header(lib, file, names, fields):
    text = header(file)
    declared = set(re.findall(r"^\s*(?:const\s+)?[a-z_][a-z_0-9]*\**\s+\**(seq_[a-z_0-9]+)\s*\(", text, re.M))
    assert declared == set(names)
    for n in declared:
        assert hasattr(lib, n), n
    body = re.search(r"typedef struct \{([^}]*)\} seq_\w+_args;", text, re.S).group(1)
    assert tuple(re.findall(r"(\w+);", body)) == fields


def _delta(S=2, T=8, Hk=2, Hv=4, Dk=16, Dv=8, dtype=B.CONV_BF16, direction=Q.SEQ_FWD, flags=D.SEQ_DELTA_QK_NORM, scale=0.0):
    return D.seq_delta_plan_create(S, T, Hk, Hv, Dk, Dv, dtype, direction, flags, scale)


def _gnorm(S=2, T=8, D=16, G=4, dtype=B.CONV_BF16, direction=Q.SEQ_FWD, flags=0, act=0, eps=1e-5):
    return N.seq_gnorm_plan_create(S, T, D, G, dtype, direction, flags, act, eps)


@pytest.mark.parametrize("make,kw,status", [
    (_delta, dict(S=0), 1), (_delta, dict(T=-1), 1), (_delta, dict(T=9), 1), (_delta, dict(Hk=0), 1), (_delta, dict(Hk=3), 1),
    (_delta, dict(Hk=8), 1), (_delta, dict(Dk=0), 1), (_delta, dict(Dv=0), 1), (_delta, dict(Dk=129), 2), (_delta, dict(Dv=1025), 2),
    (_delta, dict(Hk=1, Hv=4097, Dv=1), 2), (_delta, dict(dtype=7), 1), (_delta, dict(direction=3), 1), (_delta, dict(flags=2), 1),
    (_delta, dict(scale=float("inf")), 1), (_delta, dict(scale=float("nan")), 1), (_delta, dict(direction=Q.SEQ_STEP), 1),
    (_delta, dict(T=2, direction=Q.SEQ_STEP, flags=Q.SEQ_RAGGED), 1), (_delta, dict(S=1, T=(1 << 30) + 1), 2),
    (_delta, dict(S=1 << 22, T=1 << 22, Hk=64, Hv=64, Dv=128), 2),
    (_gnorm, dict(S=0), 1), (_gnorm, dict(T=9), 1), (_gnorm, dict(D=0), 1), (_gnorm, dict(G=0), 1), (_gnorm, dict(G=3), 1),
    (_gnorm, dict(dtype=9), 1), (_gnorm, dict(direction=Q.SEQ_STEP), 1), (_gnorm, dict(flags=2), 1), (_gnorm, dict(act=3), 1),
    (_gnorm, dict(eps=-1.0), 1), (_gnorm, dict(eps=float("nan")), 1), (_gnorm, dict(D=(1 << 20) + 1, G=1), 2),
    (_gnorm, dict(S=1 << 20, T=1 << 20, D=1 << 12, G=1 << 12), 2),
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


def test_delta_calls_check_their_arguments(lib):
    good = dict(q=P, q_ld=32, k=P, k_ld=32, v=P, v_ld=32, g=P, g_ld=4, beta=P, beta_ld=4, y=P, y_ld=32)
    st = lambda plan, name="seq_delta_fwd", **kw: _status(lib, name, plan, D.DELTA_FIELDS, **kw)      # noqa: E731
    fwd, bwd, rag, step = _delta(), _delta(direction=Q.SEQ_BWD), _delta(flags=Q.SEQ_RAGGED), _delta(T=2, direction=Q.SEQ_STEP)
    assert st(None, **good) == 1 and st(bwd, **good) == 1 and st(fwd, "seq_delta_step", **good) == 1
    for k in ("q", "k", "v", "g", "beta", "y"):
        assert st(fwd, **{**good, k: 0}) == 1, k
        assert st(fwd, **{**good, k: P + 1}) == 3, k
        assert st(fwd, **{**good, k + "_ld": 3}) == 1, k
        assert st(fwd, **{**good, k + "_ld": 1 << 31}) == 2, k
    assert st(fwd, **good, starts=P) == 1 and st(rag, **good) == 1
    assert st(fwd, **good, h_in=P, slot_count=1) == 1 and st(fwd, **good, h_out=P + 2, slot_count=2) == 3
    assert st(fwd, **good, saved=P + 4) == 3
    assert st(fwd, **good) == 4                                      # no workspace
    assert st(step, "seq_delta_step", **{**good, "q": 0}) == 1
    b = {**good, **dict(dy=P, dy_ld=32, saved=P, dq=P, dq_ld=32, dk=P, dk_ld=32, dv=P, dv_ld=32, dg=P, dg_ld=4, dbeta=P, dbeta_ld=4)}
    b.pop("y"), b.pop("y_ld")
    assert st(bwd, "seq_delta_bwd", **b) == 4
    for k in ("dy", "saved", "dq", "dk", "dv", "dg", "dbeta"):
        assert st(bwd, "seq_delta_bwd", **{**b, k: 0}) == 1, k
    assert st(bwd, "seq_delta_bwd", **b, dh_in=P, slot_count=1) == 1
    assert D.seq_delta_saved_bytes(fwd) == D.seq_delta_saved_bytes(bwd) > 0 and D.seq_delta_saved_bytes(step) == 0
    assert lib.seq_delta_saved_bytes(None) == 0 and lib.seq_delta_check(None, None) == 1
    g = _gnorm()
    assert lib.seq_delta_check(g, None) == 1 and D.seq_delta_saved_bytes(g) == 0 and st(g, **good) == 1
    for p in (fwd, bwd, rag, step, g):
        Q.seq_plan_destroy(p)


def test_gnorm_calls_check_their_arguments(lib):
    good = dict(x=P, x_ld=16, y=P, y_ld=16)
    st = lambda plan, name="seq_gnorm_fwd", **kw: _status(lib, name, plan, N.GNORM_FIELDS, **kw)      # noqa: E731
    fwd, bwd, rag = _gnorm(), _gnorm(direction=Q.SEQ_BWD), _gnorm(flags=Q.SEQ_RAGGED)
    assert st(None, **good) == 1 and st(bwd, **good) == 1
    for k in ("x", "y"):
        assert st(fwd, **{**good, k: 0}) == 1 and st(fwd, **{**good, k: P + 1}) == 3 and st(fwd, **{**good, k + "_ld": 15}) == 1, k
    for k in ("w", "b"):
        assert st(fwd, **good, **{k: P + 1}) == 3, k
    assert st(fwd, **good, stats=P + 4) == 3 and st(fwd, **good, starts=P) == 1 and st(rag, **good) == 1
    assert st(fwd, **good) == 4
    b = dict(x=P, x_ld=16, stats=P, dy=P, dy_ld=16, dx=P, dx_ld=16)
    assert st(bwd, "seq_gnorm_bwd", **b) == 4
    for k in ("x", "stats", "dy", "dx"):
        assert st(bwd, "seq_gnorm_bwd", **{**b, k: 0}) == 1, k
    assert st(bwd, "seq_gnorm_bwd", **b, dw=P) == 1 and st(bwd, "seq_gnorm_bwd", **b, db=P) == 1      # no such parameter
    for p in (fwd, bwd, rag):
        Q.seq_plan_destroy(p)


def test_python_plans_refuse_tensors_that_do_not_fit(lib):
    import torch
    p = D.SeqDeltaPlan(2, 8, 2, 4, 16, 8, B.CONV_F32)
    q, v, g = torch.zeros(8, 32), torch.zeros(8, 32), torch.zeros(8, 4)
    with pytest.raises(B.ConvError):
        p.forward(q, q, v, g, g, v)                                  # not on the GPU
    with pytest.raises(B.ConvError):
        p.step(q, q, v, g, g, None, None, v)                         # the plan's direction
    for kw in (dict(direction="sideways"), dict(scale=0.0)):
        with pytest.raises(ValueError):
            D.SeqDeltaPlan(2, 8, 2, 4, 16, 8, B.CONV_F32, **kw)
    p.close()
    n = N.SeqGroupNormPlan(2, 8, 16, 4, B.CONV_F32)
    with pytest.raises(B.ConvError):
        n.forward(torch.zeros(8, 16), torch.zeros(8, 16))
    for kw in (dict(act="tanh"), dict(direction="step")):
        with pytest.raises(ValueError):
            N.SeqGroupNormPlan(2, 8, 16, 4, B.CONV_F32, **kw)
    n.close()


# ------------------------------------------------------- the oracle's gradients against differences
def _directional(f, args, grads, name, rng, eps=1e-5):
    d = rng.standard_normal(args[name].shape)
    hi, lo = dict(args), dict(args)
    hi[name], lo[name] = args[name] + eps * d, args[name] - eps * d
    num = (f(**hi) - f(**lo)) / (2 * eps)
    ana = float((grads[name].reshape(d.shape) * d).sum())
    assert abs(num - ana) <= 2e-6 * max(1.0, abs(ana)), (name, num, ana)


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("Hk,Hv", [(2, 2), (1, 3)])
def test_delta_gradients_against_differences(norm, Hk, Hv):
    rng = np.random.default_rng(5)
    lens, Dk, Dv = [4, 0, 1, 6], 3, 5
    T, S = sum(lens), len(lens)
    n = rng.standard_normal
    a = dict(q=n((T, Hk, Dk)), k=n((T, Hk, Dk)) * 0.7, v=n((T, Hv, Dv)), g=-rng.uniform(0.05, 1, (T, Hv)), beta=rng.uniform(0, 1, (T, Hv)),
             h0=n((S, Hv, Dk, Dv)))
    dy, dh = n((T, Hv, Dv)), n((S, Hv, Dk, Dv))

    def f(**kw):
        o = R.delta(**kw, lens=lens, norm=norm)
        return float((o["y"].reshape(dy.shape) * dy).sum() + (o["h"] * dh).sum())

    g = R.delta(**a, lens=lens, norm=norm, dy=dy, dh_out=dh)
    grads = {k: g["d" + k] for k in ("q", "k", "v", "g", "beta")}
    grads["h0"] = g["dh_in"]
    for k in a:
        _directional(f, a, grads, k, rng)


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("G", [1, 2, 6])
def test_gnorm_gradients_against_differences(act, G):
    rng = np.random.default_rng(6)
    lens, D = [5, 0, 1, 7], 6
    a = dict(x=rng.standard_normal((13, D)), w=rng.standard_normal(D), b=rng.standard_normal(D))
    dy = rng.standard_normal((13, D))
    f = lambda **kw: float((R.gnorm(**kw, G=G, lens=lens, act=act, eps=1e-2)[0]["y"] * dy).sum())      # noqa: E731
    o, _ = R.gnorm(**a, G=G, lens=lens, act=act, eps=1e-2, dy=dy)
    for k in a:
        _directional(f, a, {"x": o["dx"], "w": o["dw"], "b": o["db"]}, k, rng)


@pytest.mark.parametrize("fault", ["mean", "variance", "slope", "m2"])
def test_gnorm_bounds_tell_mistakes(fault):
    """Outputs with a mistake planted leave the bounds that the kernels are held to."""
    rng = np.random.default_rng(7)
    lens, D, G, T = [9, 20], 8, 2, 29
    x, dy = rng.standard_normal((T, D)) + 0.5, rng.standard_normal((T, D))
    w, b = rng.uniform(0.5, 1.5, D), rng.standard_normal(D)
    ref, mag = R.gnorm(x, w, b, G, lens, "silu", 1e-5, dy=dy)
    wrong = {k: v.copy() for k, v in ref.items()}
    if fault == "mean":
        wrong["y"] = R.gnorm(x, w, b, G, [29], "silu", 1e-5)[0]["y"]              # over both sequences
    elif fault == "variance":
        wrong["y"] = R.gnorm(x * np.sqrt(8 / 9), w, b, G, lens, "silu", 1e-3)[0]["y"]
    elif fault == "slope":
        wrong["dx"] = R.gnorm(x, w, b, G, lens, "gelu", 1e-5, dy=dy)[0]["dx"]
    else:
        wrong["dx"] = ref["dx"] + 1e-3
    with pytest.raises(AssertionError):
        for k in ("y", "dx"):
            R.O.check(k, wrong[k], ref[k], mag[k], 400, False)


@pytest.mark.parametrize("fault", ["decay", "order", "shared"])
def test_delta_bounds_tell_mistakes(fault):
    rng = np.random.default_rng(8)
    T, H, K, V = 150, 2, 8, 6
    q, k, v = rng.standard_normal((T, H, K)), rng.standard_normal((T, H, K)), rng.standard_normal((T, H, V))
    g, beta = -rng.uniform(0, 0.1, (T, H)), rng.uniform(0, 1, (T, H))
    h0 = rng.standard_normal((1, H, K, V))
    ref = R.delta(q, k, v, g, beta, [T], h0, True)
    g2, k2, b2 = g.copy(), k, beta
    if fault == "decay":
        g2[64] = 0                                  # the first token of a chunk does not decay
    elif fault == "order":
        b2 = beta.copy()
        b2[[100, 101]] = beta[[101, 100]]
    else:
        k2 = k[:, [1, 0]]
    wrong = R.delta(q, k2, v, g2, b2, [T], h0, True)
    with pytest.raises(AssertionError):
        R.check_heads("y", wrong["y"], ref["y"], H, False, R.FORWARD)
