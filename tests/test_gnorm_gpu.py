"""The group norm with an activation on the GPU against the 64-bit oracle, element by element, within bounds counted
from its operations: group layouts, lengths, strides, values and masks of any size, both types, both directions."""
import numpy as np
import pytest

from convolution_forward_implicit_gb300 import gnorm as N
from convolution_forward_implicit_gb300.binding import CONV_BF16, CONV_F32
from tests import delta_oracle as R
from tests.test_seq_gpu import Box, host, starts_of

pytestmark = pytest.mark.gpu
CODE = {False: CONV_F32, True: CONV_BF16}
K = 400              # operations on the longest way: sums of up to 300 terms, the functions of a value


def run(c, b, bf16, x, w, bias, dy, lens, D, G, act, ragged, eps=1e-5, pad=0, in_place=False):
    import torch
    S, T = len(lens), sum(lens)
    starts = starts_of(lens) if ragged else None
    y, stats = b.out(T, D, pad=pad), b.out(S, G, 2, dtype=torch.float32)
    fwd = N.SeqGroupNormPlan(S, T, D, G, CODE[bf16], "fwd", ragged=ragged, act=act, eps=eps).allocate()
    fwd.workspace.fill_(0xFF)
    fwd.forward(x, y, w=w, b=bias, starts=starts, stats=stats)
    y2 = b.out(T, D, pad=pad)
    fwd.forward(x, y2, w=w, b=bias, starts=starts)          # without statistics: the same
    assert bool((y == y2).all())
    out = dict(y=y, stats=stats)
    if dy is not None:
        bwd = N.SeqGroupNormPlan(S, T, D, G, CODE[bf16], "bwd", ragged=ragged, act=act, eps=eps).allocate()
        bwd.workspace.fill_(0xFF)
        f32 = torch.float32
        out.update(dx=b.out(T, D, pad=pad), dw=b.out(D, dtype=f32) if w is not None else None, db=b.out(D, dtype=f32) if bias is not None else None)
        bwd.backward(x, stats, dy, out["dx"], w=w, b=bias, dw=out["dw"], db=out["db"], starts=starts)
        dx = b.out(T, D, pad=pad)
        bwd.backward(x, stats, dy, dx, w=w, b=bias, starts=starts)         # no parameters' gradients: the same
        assert bool((dx == out["dx"]).all())
    b.check_guards()
    return out


def compare(out, ref, mag, bf16, terms=0, k=K):
    for name in ("y", "dx", "dw", "db"):
        if out.get(name) is not None:
            R.O.check(name, host(out[name]), ref[name], mag[name], k + (terms if name in ("dw", "db") else 0), bf16 and name in ("y", "dx"))


UNIFORM = [[1], [2] * 3, [300], [49] * 4, [1] * 5]
RAGGED = [[0, 1, 0, 0, 5, 2, 0], [3, 140, 1, 17], [0], [0, 0], [257, 2, 64]]
WIDTHS = [(8, 1), (16, 4), (24, 24), (77, 7), (96, 3), (264, 33), (1, 1), (520, 2), (1030, 5)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("lens,ragged", [(v, False) for v in UNIFORM] + [(v, True) for v in RAGGED])
@pytest.mark.parametrize("D,G", WIDTHS)
def test_gnorm(bf16, lens, ragged, D, G):
    S, T = len(lens), sum(lens)
    act = ["none", "silu", "gelu"][(D + T) % 3]
    pad = [0, 8, 3][(D + S) % 3]
    b = Box(D + 31 * T, bf16)
    x, xe = b.put(b.rng.standard_normal((T, D)) * 2 + b.rng.standard_normal(D), pad=pad)
    w, we = b.put(b.rng.uniform(0.5, 1.5, D))
    bias, be = b.normal(D, std=0.3)
    dy, dye = b.normal(T, D, pad=pad)
    if (D + S) % 4 == 0:
        w, we = None, None
    if (D + S) % 5 == 0:
        bias, be = None, None
    eps = 1e-3
    out = run(None, b, bf16, x, w, bias, dy, lens, D, G, act, ragged, eps=eps, pad=pad)
    ref, mag = R.gnorm(xe, we, be, G, lens, act, eps, dy=dye)
    compare(out, ref, mag, bf16, terms=T)
    st = host(out["stats"])
    for s, n in enumerate(lens):
        if n == 0:
            assert (st[s] == 0).all()
        else:
            assert np.allclose(st[s, :, 1], ref["stats"][s, :, 1], rtol=1e-4) and np.allclose(st[s, :, 0], ref["stats"][s, :, 0], atol=1e-5 * 4)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("S,T,D,G", [(2, 6000, 64, 8), (1, 9001, 40, 5), (3, 3 * 2100, 136, 136), (1, 700, 4096, 4), (2, 60, 16384, 1),
                                     (2, 8, 10240, 10240), (1, 40, 6145, 5 * 1229)])
def test_long_and_wide(bf16, S, T, D, G):
    """Many slabs of tokens, many blocks of channels, groups that lie in several of them."""
    b = Box(S + T + D, bf16)
    x, xe = b.put(b.rng.standard_normal((T, D)) + 0.5)
    w, we = b.put(b.rng.uniform(0.5, 1.5, D))
    bias, be = b.normal(D, std=0.3)
    dy, dye = b.normal(T, D)
    out = run(None, b, bf16, x, w, bias, dy, [T // S] * S, D, G, "silu", False)
    ref, mag = R.gnorm(xe, we, be, G, [T // S] * S, "silu", 1e-5, dy=dye)
    compare(out, ref, mag, bf16, terms=T)


@pytest.mark.parametrize("mean", [0.0, 100.0, -3000.0])
@pytest.mark.parametrize("G", [2, 16])
def test_means_far_from_zero(mean, G):
    """The variance comes from differences, however far the mean lies; the error goes with x less mean alone."""
    b = Box(int(abs(mean)) + G, False)
    T, D = 900, 32
    x, xe = b.put(b.rng.standard_normal((T, D)) + mean)
    out = run(None, b, False, x, None, None, None, [450, 450], D, G, "none", False)
    ref, mag = R.gnorm(xe, None, None, G, [450, 450], "none", 1e-5)
    compare(out, ref, mag, False, k=8)


def test_constant_rows_and_one_value():
    """No variance: rstd is 1 / sqrt(eps), y is b; the gradient's sums vanish."""
    import torch
    b = Box(3, False)
    x = torch.full((50, 16), 7.25, device="cuda")
    bias, be = b.normal(16)
    y, stats = b.out(50, 16), b.out(2, 4, 2, dtype=torch.float32)
    N.SeqGroupNormPlan(2, 50, 16, 4, CONV_F32, eps=1e-4).forward(x, y, b=bias, stats=stats)
    assert bool((y == bias).all()) and bool((stats[..., 0] == 7.25).all()) and np.allclose(host(stats)[..., 1], 100.0, rtol=1e-6)


@pytest.mark.parametrize("bf16", [False, True])
def test_rows_at_any_element(bf16):
    b = Box(5, bf16)
    T, D, G = 90, 48, 6
    a = b.rng.standard_normal((T, D))
    dy0 = b.rng.standard_normal((T, D))
    for shift, pad in [(0, 0), (1, 0), (2, 2), (1, 1), (0, 4)]:
        x, xe = b.put(a, pad=pad, shift=shift)
        dy, dye = b.put(dy0, pad=pad, shift=shift)
        out = run(None, b, bf16, x, None, None, dy, [30] * 3, D, G, "gelu", False, pad=pad)
        ref, mag = R.gnorm(xe, None, None, G, [30] * 3, "gelu", 1e-5, dy=dye)
        compare(out, ref, mag, bf16, terms=T)


def test_in_place():
    """y may be x, and dx may be dy."""
    import torch
    b = Box(6, True)
    x, _ = b.normal(700, 128)
    dy, _ = b.normal(700, 128)
    y, stats, dx = b.out(700, 128), b.out(2, 8, 2, dtype=torch.float32), b.out(700, 128)
    fwd, bwd = (N.SeqGroupNormPlan(2, 700, 128, 8, CONV_BF16, d, act="silu") for d in ("fwd", "bwd"))
    fwd.forward(x, y, stats=stats)
    bwd.backward(x, stats, dy, dx)
    x2, dy2 = x.clone(), dy.clone()
    bwd.backward(x, stats, dy2, dy2)
    fwd.forward(x2, x2)
    assert torch.equal(x2, y) and torch.equal(dy2, dx)


def test_bad_values_stay_in_their_sequence_and_group():
    import torch
    b = Box(7, False)
    x, _ = b.normal(90, 32)
    dy, _ = b.normal(90, 32)
    clean = run(None, b, False, x, None, None, dy, [30] * 3, 32, 4, "silu", False)
    x[40, 9], x[41, 10] = float("nan"), float("inf")           # sequence 1, group 1
    bad = run_raw(x, dy)
    for name in ("y", "dx"):
        keep = torch.ones(90, 32, dtype=torch.bool, device="cuda")
        keep[30:60, 8:16] = False
        assert torch.equal(bad[name][keep], clean[name][keep])
        assert bool(torch.isnan(bad[name][30:60, 8:16]).all())


def run_raw(x, dy):
    import torch
    y, stats, dx = torch.empty_like(x), torch.empty(3, 4, 2, device="cuda"), torch.empty_like(x)
    N.SeqGroupNormPlan(3, 90, 32, 4, CONV_F32, act="silu").forward(x, y, stats=stats)
    N.SeqGroupNormPlan(3, 90, 32, 4, CONV_F32, "bwd", act="silu").backward(x, stats, dy, dx)
    return dict(y=y, dx=dx)


def test_many_sequences_and_large_offsets():
    import torch
    # more sequences than a launch's second dimension holds
    S = 70000
    x = torch.randn(2 * S, 8, device="cuda")
    y = torch.empty_like(x)
    N.SeqGroupNormPlan(S, 2 * S, 8, 2, CONV_F32).forward(x, y)
    v = x.double().view(S, 2, 2, 4)
    ref = (v - v.mean((1, 3), keepdim=True)) / torch.sqrt(v.var((1, 3), unbiased=False, keepdim=True) + 1e-5)
    assert float((y.double() - ref.view_as(x)).abs().max()) < 1e-4       # (8 values: rstd up to 300, x up to 5)
    # tokens beyond 2^31 elements
    ld = 1 << 22
    wide = torch.empty(599 * ld + 64, dtype=torch.bfloat16, device="cuda")
    a, o = wide.as_strided((600, 32), (ld, 1), 0), wide.as_strided((600, 32), (ld, 1), 32)
    small = torch.randn(600, 32, device="cuda").bfloat16()
    a.copy_(small)
    p, want = N.SeqGroupNormPlan(2, 600, 32, 4, CONV_BF16, act="silu"), torch.empty(600, 32, dtype=torch.bfloat16, device="cuda")
    p.forward(small, want)
    p.forward(a, o)
    assert torch.equal(o, want)


def test_bounds_outside_their_contract():
    import torch
    b = Box(9, False)
    x, _ = b.normal(170, 24)
    dy, _ = b.normal(170, 24)
    for bad in ([0, 500, -7, 170], [0, 100, 20, 170], [90, 10, 5, 2], [0, 0, 0, 0]):
        st = torch.tensor(bad, dtype=torch.int32, device="cuda")
        y, stats, dx = b.out(170, 24), b.out(3, 3, 2, dtype=torch.float32), b.out(170, 24)
        N.SeqGroupNormPlan(3, 170, 24, 3, CONV_F32, ragged=True, act="gelu").forward(x, y, starts=st, stats=stats)
        N.SeqGroupNormPlan(3, 170, 24, 3, CONV_F32, "bwd", ragged=True, act="gelu").backward(x, stats, dy, dx, starts=st)
        b.check_guards()


def test_streams_and_graphs():
    import torch
    b = Box(10, True)
    x, _ = b.normal(1500, 384)
    w, _ = b.put(b.rng.uniform(0.5, 1.5, 384))
    dy, _ = b.normal(1500, 384)
    fwd, bwd = (N.SeqGroupNormPlan(3, 1500, 384, 32, CONV_BF16, d, act="silu") for d in ("fwd", "bwd"))
    y, stats, dx, dw = b.out(1500, 384), b.out(3, 32, 2, dtype=torch.float32), b.out(1500, 384), b.out(384, dtype=torch.float32)

    def call(**kw):
        fwd.forward(x, y, w=w, stats=stats, **kw)
        bwd.backward(x, stats, dy, dx, w=w, dw=dw, **kw)

    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, stats, dx, dw)]

    def same():
        torch.cuda.synchronize()
        for t, u in zip((y, stats, dx, dw), want):
            assert torch.equal(t, u)
            t.fill_(2.0)

    side = torch.cuda.Stream()
    same()
    call(stream=side.cuda_stream)
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        graph.replay()
        same()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("lens,ragged", [([1] * 7, False), ([1, 3, 0, 1, 200, 1], True)])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_groups_of_one_value_pass_no_gradient(bf16, lens, ragged, act):
    """A token by itself and as many groups as channels: the value is its mean, so dx is zero, exactly; the others as ever."""
    import torch
    D, T = 384, sum(lens)
    b = Box(D + T, bf16)
    x, xe = b.normal(T, D)
    w, we = b.put(b.rng.uniform(0.5, 1.5, D))
    bias, be = b.normal(D, std=0.3)
    dy, dye = b.normal(T, D)
    out = run(None, b, bf16, x, w, bias, dy, lens, D, D, act, ragged)
    at = np.cumsum([0] + list(lens))
    for s, n in enumerate(lens):
        if n == 1:
            assert bool((out["dx"][at[s]] == 0).all())
    ref, mag = R.gnorm(xe, we, be, D, lens, act, 1e-5, dy=dye)
    compare(out, ref, mag, bf16, terms=T)
    # a value that is not finite still shows in its own place, and there only
    dy[0, 5] = float("nan")
    bad = b.out(T, D)
    N.SeqGroupNormPlan(len(lens), T, D, D, CODE[bf16], "bwd", ragged=ragged, act=act).backward(
        x, out["stats"], dy, bad, w=w, b=bias, starts=starts_of(lens) if ragged else None)
    assert bool(torch.isnan(bad[0, 5])) and int(torch.isnan(bad.float()).sum()) == 1
