"""The sequence-mixing operators on tensors beyond 2^31 elements (2.17e9, 4.3 GB each in bf16), so that offsets need
64 bits, forward and backward.  The oracle checks the tokens around element 2^31 and the last ones, from windows of the inputs."""
import numpy as np
import pytest

from convolution_forward_implicit_gb300 import seq as Q
from convolution_forward_implicit_gb300.binding import CONV_BF16
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
