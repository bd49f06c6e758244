"""The sequence-mixing operators on tensors beyond 2^31 elements (2.17e9, 4.3 GB each in bf16), so that offsets need
64 bits, forward and backward: the oracle checks the tokens around element 2^31 and the last ones, from windows of the
inputs.  And more sequences, channels and groups than a launch's grid has places in one dimension."""
import numpy as np
import pytest

from convolution_forward_implicit_gb300 import seq as Q
from convolution_forward_implicit_gb300.binding import CONV_BF16, CONV_F32
from tests import seq_oracle as O

pytestmark = pytest.mark.gpu
D, L = 4096, 265_000
T, WRAP = 2 * L, (1 << 31) // 4096           # two sequences; the token with element 2^31
CHECK = 48


@pytest.fixture(autouse=True)
def memory():
    import torch
    yield
    torch.cuda.empty_cache()


def host(t):
    return t.double().cpu().numpy()


def normal(seed, *shape):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)


def check(name, got, ref, mag, k):
    O.check(name, host(got), ref, mag, k, True)


def test_convolution():
    import torch
    assert T * D > 1 << 31 and L < WRAP < T - CHECK
    W = 4
    x, dy, w, bias = normal(1, T, D), normal(2, T, D), normal(3, D, W), normal(4, D)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dw, db, state = torch.empty(D, W, device="cuda"), torch.empty(D, device="cuda"), torch.empty(2, W - 1, D, dtype=torch.bfloat16, device="cuda")
    Q.SeqConvPlan(2, T, D, W, CONV_BF16).forward(x, w, bias, y, state_out=state)
    Q.SeqConvPlan(2, T, D, W, CONV_BF16, "bwd").backward(x, w, bias, dy, dx, dw, db)
    assert torch.equal(state[1], x[-(W - 1):])
    for a, b in ((WRAP - CHECK, WRAP + CHECK), (T - CHECK, T)):
        head = host(x[a - W + 1:a])[None]
        args = [host(x[a:b]), host(w), host(bias), [b - a], head]
        ref, _, mag = O.conv(*args)
        check("y", y[a:b], ref, mag, W + 100)
        ref, mag = O.conv_grad(*args, host(dy[a:b]))
        n = b - a if b == T else b - a - W + 1       # (the last ones take from the tokens behind the window)
        check("dx", dx[a:a + n], ref["dx"][:n], mag["dx"][:n], W + 100)


def test_scan():
    """States of this A and these steps forget all but 1e-12 in 400 tokens: windows start from nothing so far away."""
    import torch
    N, FAR = 4, 400
    x, dt, dy, B, C = normal(1, T, D), normal(2, T, D), normal(3, T, D), normal(4, T, N), normal(5, T, N)
    A = -(torch.rand(D, N, device="cuda") * 3 + 0.3)
    y, dx, ddt, dB, dC = (torch.empty_like(t) for t in (x, x, x, B, C))
    p, q = Q.SeqScanPlan(2, T, D, N, CONV_BF16), Q.SeqScanPlan(2, T, D, N, CONV_BF16, "bwd")
    saved = q.allocate_saved()
    p.forward(x, dt, A, B, C, y, saved=saved)
    q.backward(x, dt, A, B, C, dy, saved, dx, ddt, torch.empty_like(A), dB, dC)
    ch = torch.tensor([0, 1, 7, 2047, 2048, 4090, 4095], device="cuda")
    k = 4 * 2 * FAR + N + 100
    for a, b in ((WRAP - CHECK, WRAP + CHECK), (T - CHECK, T)):
        lo, hi = a - FAR, min(b + FAR, T)
        part = lambda t: host(t[lo:hi][:, ch])      # noqa: E731
        ref, mag = O.scan(part(x), part(dt), host(A[ch]), host(B[lo:hi]), host(C[lo:hi]), 1, [hi - lo], np.zeros((1, len(ch), N)), dy=part(dy))
        for name, t, more in (("y", y, 0), ("dx", dx, k), ("ddt", ddt, k)):
            check(name, t[a:b][:, ch], ref[name][FAR:FAR + b - a], mag[name][FAR:FAR + b - a], k + more)


def test_norm():
    import torch
    x, res, dy, dro, w = normal(1, T, D), normal(2, T, D), normal(3, T, D), normal(4, T, D), normal(5, D)
    y, ro, dx, dres = (torch.empty_like(x) for _ in range(4))
    dw = torch.empty(D, device="cuda")
    Q.SeqNormPlan(T, D, CONV_BF16, res_dtype=CONV_BF16).forward(x, y=y, res=res, res_out=ro, w_pre=w)
    Q.SeqNormPlan(T, D, CONV_BF16, "bwd", res_dtype=CONV_BF16).backward(x, dx, dy=dy, dres_out=dro, res=res, w_pre=w, dres=dres, dw_pre=dw)
    k = D / 32 + 120
    for a, b in ((WRAP - 4, WRAP + 4), (T - 8, T)):
        ref, mag = O.norm(host(x[a:b]), False, 1e-5, False, True, res=host(res[a:b]), w_pre=host(w), dy=host(dy[a:b]), dres_out=host(dro[a:b]))
        for name, t, times in (("y", y, 1), ("res_out", ro, 1), ("dx", dx, 2), ("dres", dres, 2)):
            check(name, t[a:b], ref[name], mag[name], times * k)


# ------------------------------------------------ more sequences, channels and groups than a grid's dimensions
def f32(rng, *shape, std=1.0):
    import torch
    a = (rng.standard_normal(shape) * std).astype(np.float32)
    return torch.from_numpy(a).cuda(), a.astype(np.float64)


def near(name, got, ref, mag, k):
    O.check(name, host(got), ref, mag, k, False)


def test_many_sequences():
    """Prompts of none to two tokens and steps, of more sequences than 32768 blocks or 65535."""
    import torch
    rng = np.random.default_rng(1)
    S, D_, N, W = 70_001, 5, 3, 3
    lens = rng.integers(0, 3, S)
    T_ = int(lens.sum())
    starts = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    (x, xe), (w, we), (bias, be), (state, se) = f32(rng, T_, D_), f32(rng, D_, W), f32(rng, D_), f32(rng, S, W - 1, D_)
    y, left = torch.empty_like(x), torch.empty_like(state)
    Q.SeqConvPlan(S, T_, D_, W, CONV_F32, ragged=True).forward(x, w, bias, y, starts=starts, state_in=state, state_out=left)
    ref, refl, mag = O.conv(xe, we, be, lens, se)
    near("conv y", y, ref, mag, W + 100)
    assert np.array_equal(host(left), refl)
    (x1, x1e), y1 = f32(rng, S, D_), torch.empty(S, D_, device="cuda")
    Q.SeqConvPlan(S, S, D_, W, CONV_F32, "step").step(x1, w, bias, left, left, y1)
    win = np.concatenate([refl, x1e[:, None]], 1)
    pre = be + (win * we.T).sum(1)
    near("conv step y", y1, O.silu(pre), 1.1 * (np.abs(be) + np.abs(win * we.T).sum(1)), W + 100)
    assert np.array_equal(host(left), win[:, 1:])

    (dt, dte), (B, Be), (C, Ce), (h, he) = f32(rng, T_, D_), f32(rng, T_, N), f32(rng, T_, N), f32(rng, S, D_, N)
    A = -torch.rand(D_, N, device="cuda") - 0.2
    y, hl = torch.empty_like(x), torch.empty_like(h)
    p, q = (Q.SeqScanPlan(S, T_, D_, N, CONV_F32, d, ragged=True) for d in ("fwd", "bwd"))
    saved = q.allocate_saved()
    p.forward(x, dt, A, B, C, y, starts=starts, h_in=h, h_out=hl, saved=saved)
    (dy, dye), (dh, dhe) = f32(rng, T_, D_), f32(rng, S, D_, N)
    g = dict(dx=torch.empty_like(x), ddt=torch.empty_like(x), dA=torch.empty_like(A), dB=torch.empty_like(B), dC=torch.empty_like(C), dh_in=torch.empty_like(h))
    q.backward(x, dt, A, B, C, dy, saved, starts=starts, h_in=h, dh_out=dh, **g)
    ref, mag = O.scan(xe, dte, host(A), Be, Ce, 1, lens, he, dy=dye, dh_out=dhe)
    near("scan y", y, ref["y"], mag["y"], N + 120)
    near("h", hl, ref["h"], mag["h"], N + 120)
    for name, v in g.items():
        near(name, v, ref[name], mag[name], 2 * N + 240 + (T_ if name == "dA" else D_))
    S2 = 140_003                                  # four sequences a thread
    t = [f32(rng, S2, n) for n in (D_, D_, N, N)]
    (h, he), y1 = f32(rng, S2, D_, N), torch.empty(S2, D_, device="cuda")
    Q.SeqScanPlan(S2, S2, D_, N, CONV_F32, "step").step(t[0][0], t[1][0], A, t[2][0], t[3][0], h, h, y1)
    delta = O.softplus(t[1][1])
    u = (delta * t[0][1])[:, :, None] * t[2][1][:, None]
    new, mag = np.exp(delta[:, :, None] * host(A)) * he + u, np.exp(delta[:, :, None] * host(A)) * np.abs(he) + np.abs(u)
    near("step h", h, new, mag, 120)
    near("step y", y1, (new * t[3][1][:, None]).sum(-1), (mag * np.abs(t[3][1][:, None])).sum(-1), N + 120)


@pytest.mark.parametrize("W_,G", [((1 << 22) - 3, 1), (1 << 22, 1), (1 << 22, 1 << 15), (32513 * 129, 32513)])
def test_the_widest_scans(W_, G):
    """2^22 channels, 2^15 groups, and groups just wider than a block."""
    import torch
    rng = np.random.default_rng(2)
    N, lens = 2, [2, 1]
    (x, xe), (dt, dte), (dy, dye) = (f32(rng, 3, W_) for _ in range(3))
    (B, Be), (C, Ce), (h, he) = f32(rng, 3, G * N), f32(rng, 3, G * N), f32(rng, 2, W_, N)
    A = -torch.rand(W_, N, device="cuda") - 0.2
    starts = torch.tensor([0, 2, 3], dtype=torch.int32, device="cuda")
    p, q = (Q.SeqScanPlan(2, 3, W_, N, CONV_F32, d, G=G, ragged=True) for d in ("fwd", "bwd"))
    y, hl, saved = torch.empty_like(x), torch.empty_like(h), q.allocate_saved()
    p.forward(x, dt, A, B, C, y, starts=starts, h_in=h, h_out=hl, saved=saved)
    g = dict(dx=torch.empty_like(x), ddt=torch.empty_like(x), dA=torch.empty_like(A), dB=torch.empty_like(B), dC=torch.empty_like(C))
    q.backward(x, dt, A, B, C, dy, saved, starts=starts, h_in=h, **g)
    ref, mag = O.scan(xe, dte, host(A), Be, Ce, G, lens, he, dy=dye)
    near("y", y, ref["y"], mag["y"], N + 120)
    near("h", hl, ref["h"], mag["h"], N + 120)
    for name, v in g.items():
        near(name, v, ref[name], mag[name], 2 * N + 240 + W_ // G)
    ((x1, x1e), (d1, d1e)), ((b1, b1e), (c1, c1e)) = (f32(rng, 1, W_) for _ in range(2)), (f32(rng, 1, G * N) for _ in range(2))
    y1, h1 = torch.empty_like(x1), h[:1].clone()
    Q.SeqScanPlan(1, 1, W_, N, CONV_F32, "step", G=G).step(x1, d1, A, b1, c1, h1, h1, y1)
    ref, mag = O.scan(x1e, d1e, host(A), b1e, c1e, G, [1], he[:1])
    near("step y", y1, ref["y"], mag["y"], N + 120)
    near("step h", h1, ref["h"], mag["h"], N + 120)


def test_the_widest_convolutions():
    import torch
    rng = np.random.default_rng(3)
    W = 2
    for D_ in ((1 << 22) - 3, 1 << 22):
        (x, xe), (w, we), (bias, be), (state, se) = f32(rng, 3, D_), f32(rng, D_, W), f32(rng, D_), f32(rng, 3, 1, D_)
        y, left = torch.empty_like(x), torch.empty(3, 1, D_, device="cuda")
        Q.SeqConvPlan(1, 3, D_, W, CONV_F32).forward(x, w, bias, y, state_in=state[:1], state_out=left[:1])
        ref, refl, mag = O.conv(xe, we, be, [3], se[:1])
        near("y", y, ref, mag, W + 100)
        assert np.array_equal(host(left[:1]), refl)
        Q.SeqConvPlan(3, 3, D_, W, CONV_F32, "step").step(x, w, bias, state, left, y)
        ref, refl, mag = O.conv(xe, we, be, [1, 1, 1], se)
        near("step", y, ref, mag, W + 100)
        assert np.array_equal(host(left), refl)
