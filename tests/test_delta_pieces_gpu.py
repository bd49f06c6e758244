"""The delta rule over long sequences whose axis is cut for the walk: what passes through a piece, and many sequences in one call."""
import numpy as np
import pytest

from convolution_forward_implicit_gb300 import delta as D
from convolution_forward_implicit_gb300 import seq as Q
from tests import delta_oracle as R
from tests.test_delta_gpu import CODE, Case
from tests.test_seq_gpu import Box, host, slots_of

pytestmark = pytest.mark.gpu


def pieces(plan):
    return int(Q.seq_plan_describe(plan.handle).split("piece_chunks=")[1])


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 64), (32, 24)])
def test_nothing_grows_from_nothing(bf16, shift, Dk, Dv):
    """Keys longer than 1 let a state grow, beyond fp32's range over a piece of the axis; a column of values that are zero, from a state
    of zero, stays zero all the same, and a key that no state has met passes nothing on."""
    import torch
    b = Box(Dk + shift, bf16)
    T, H = 2200, 1
    k = np.zeros((T, Dk))
    k[:, 0] = 1.75                                    # 1 - k^2 = -2.0625 a token: 2^67 a chunk, beyond the range after two
    k, _ = b.put(k, shift=shift, pad=8 * shift)
    q, _ = b.normal(T, Dk, shift=shift, pad=8 * shift)
    v = b.rng.standard_normal((T, H * Dv))
    v[:, ::3] = 0
    v[:, 1::3] = 0
    v, _ = b.put(v, shift=shift, pad=8 * shift)
    g, beta = torch.zeros(T, H, device="cuda"), torch.ones(T, H, device="cuda")
    h0 = np.zeros((1, H, Dk, Dv))
    h0[:, :, 1:, 1::3] = b.rng.standard_normal(h0[:, :, 1:, 1::3].shape)
    h_in, he = b.put(h0, dtype=torch.float32)
    plan = D.SeqDeltaPlan(1, T, H, H, Dk, Dv, CODE[bf16], qk_norm=False)
    assert pieces(plan) > 0
    y, h = b.out(T, H * Dv), b.out(1, H, Dk, Dv, dtype=torch.float32)
    plan.forward(q, k, v, g, beta, y, h_in=h_in, h_out=h)
    assert bool((y[:, ::3] == 0).all()) and bool((h[..., ::3] == 0).all())
    # rows that no key reaches stay as they were, and are read
    assert bool((h[..., 1::3] == h_in[..., 1::3]).all())
    want = (host(q) @ he[0, 0])[:, 1::3] / np.sqrt(Dk)
    R.check("y", host(y)[:, 1::3], want, bf16, R.FORWARD)
    # the others grow beyond all bounds
    assert not bool(torch.isfinite(h[..., 2::3]).all())
    plan.check()
    b.check_guards()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("lens", [[64] * 40, [1] * 100 + [1500] + [70] * 20 + [0] * 30 + [900], [0] * 50 + [2300] + [0] * 50, [1400] + [1] * 300,
                                  [1] * 20 + [3000, 0, 3300, 99], [0, 1800, 2] * 3 + [700]])
def test_few_long_sequences_among_many(bf16, lens):
    """The plan does not know where the tokens are.  In place of the states, too."""
    c = Case(len(lens), bf16, lens, 1, 1, 64, 64, True, decay=0.02)
    at, sl = slots_of(c.S, c.b.rng, c.S + 2, [0, c.S // 2])
    h_in, full = c.b.normal(c.S + 2, 1, 64, 64, std=0.3, dtype=c.f32)
    h0 = np.where((at >= 0)[:, None, None, None], full[at], 0)
    ref = R.delta(**c.exact, lens=lens, h0=h0, norm=True)
    fwd, y, h = c.plan("fwd").allocate(), c.b.out(c.T, 64), c.b.out(c.S + 2, 1, 64, 64, dtype=c.f32)
    fwd.workspace.fill_(0xFF)
    fwd.forward(*c.ins(), y, starts=c.starts, h_in=h_in, h_out=h, slots=sl)
    c.check(dict(y=y), ref)
    c.check_states("h", h, ref["h"], at, R.FORWARD)
    fwd.check()
    c.b.check_guards()
    both, y2 = h_in.clone(), c.b.out(c.T, 64)
    fwd.forward(*c.ins(), y2, starts=c.starts, h_in=both, h_out=both, slots=sl)
    assert bool((y2 == y).all()) and np.array_equal(host(both)[at[at >= 0]], host(h)[at[at >= 0]])
    assert (pieces(fwd) > 0) == (max(lens) in (3300, 1800))
