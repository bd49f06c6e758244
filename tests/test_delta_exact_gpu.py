"""The delta rule on the GPU where products are exact: keys that are unit vectors, beta 1, no decay.  A token then replaces one row
of the state by its value and reads it back, so that large states cancel and what the products leave of them shows."""
import numpy as np
import pytest

from convolution_forward_implicit_gb300 import delta as D
from tests.test_delta_gpu import CODE
from tests.test_seq_gpu import Box, host

pytestmark = pytest.mark.gpu
LARGE = 2.0 ** 20


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (128, 200), (40, 24)])
def test_large_states_that_are_overwritten(bf16, Dk, Dv):
    """h'^T k is a row of h_in, r; u = v - r, y = r + u and the row left is r + u.  In bf16 r and u are carried in 24 bits: u is rounded once, by half a
    step of values below 2 LARGE, 2^-24 2 LARGE, and y and the row are off by that (y by its own rounding too).  In fp32 an
    operand is two tf32 parts, which leave 2^-22 of a product: r twice, u twice.  The gradient at a row of h_in is dh + dy - (dh + dy), with
    the same roundings."""
    import torch
    b = Box(Dk + Dv, bf16)
    T, H = Dk, 2
    order = b.rng.permutation(Dk)
    unit = np.zeros((T, H, Dk))
    unit[np.arange(T), :, order] = 1
    q, _ = b.put(unit.reshape(T, -1))
    v, ve = b.normal(T, H * Dv)
    dy, _ = b.normal(T, H * Dv)
    f32 = torch.float32
    g, beta = torch.zeros(T, H, device="cuda"), torch.ones(T, H, device="cuda")
    large = lambda: b.put(b.rng.uniform(0.5, 1, (1, H, Dk, Dv)) * b.rng.choice([-1, 1], (1, H, Dk, Dv)) * LARGE, dtype=f32)[0]      # noqa: E731
    h_in, dh_out = large(), large()
    fwd, bwd = (D.SeqDeltaPlan(1, T, H, H, Dk, Dv, CODE[bf16], d, qk_norm=False, scale=1.0) for d in ("fwd", "bwd"))
    y, h, saved = b.out(T, H * Dv), b.out(1, H, Dk, Dv, dtype=f32), bwd.allocate_saved()
    fwd.forward(q, q, v, g, beta, y, h_in=h_in, h_out=h, saved=saved)
    off = 2.0 ** -24 * 2 * LARGE if bf16 else 4 * 2.0 ** -22 * 2 * LARGE
    want = ve.reshape(T, H, Dv)
    assert (np.abs(host(y).reshape(want.shape) - want) <= off + (2.0 ** -8 * (np.abs(want) + off) if bf16 else 0)).all()
    rows = np.zeros((H, Dk, Dv))
    rows[:, order] = want.transpose(1, 0, 2)
    assert (np.abs(host(h)[0] - rows) <= off).all()
    d = [torch.empty_like(t) for t in (q, q, v, g, beta)]
    dh_in = b.out(1, H, Dk, Dv, dtype=f32)
    bwd.backward(q, q, v, g, beta, dy, saved, *d, dh_out=dh_out, dh_in=dh_in)
    assert (np.abs(host(dh_in)) <= 2 * off).all()
    fwd.check()
    b.check_guards()
