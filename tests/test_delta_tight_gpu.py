"""fp32 results of the delta rule within bounds that a lost low part of an operand leaves (tests/test_delta_tight.py has the bounds and shows that)."""
import numpy as np
import pytest

from tests import delta_oracle as R
from tests.test_delta_gpu import Case
from tests.test_delta_tight import BACKWARD, FORWARD
from tests.test_seq_gpu import host

pytestmark = pytest.mark.gpu
CASES = [([300], False, 1, 1, 128, 128), ([129, 3, 63, 128], True, 2, 4, 64, 64), ([200, 77], True, 1, 3, 37, 19), ([2000], False, 1, 2, 128, 128),
         ([1500] * 2, False, 1, 2, 64, 64), ([500] * 4, False, 2, 2, 96, 200), ([190], False, 1, 2, 128, 36)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("lens,ragged,Hk,Hv,Dk,Dv", CASES)
def test_results_in_24_bits(bf16, lens, ragged, Hk, Hv, Dk, Dv):
    """Outputs, states and gradients in fp32; of bf16 calls what they leave in fp32."""
    c = Case(3 * Dk + Dv, bf16, lens, Hk, Hv, Dk, Dv, ragged, decay=0.05)
    h_in, h0, at, sl = c.states()
    dh_out, _ = c.b.normal(c.S + 2, Hv, Dk, Dv, dtype=c.f32)
    ref = R.delta(**c.exact, lens=lens, h0=h0, norm=True, dy=c.dye.reshape(c.T, Hv, Dv), dh_out=host(dh_out)[at])
    y, h, dh = c.b.out(c.T, Hv * Dv), c.b.out(c.S + 2, Hv, Dk, Dv, dtype=c.f32), c.b.out(c.S + 2, Hv, Dk, Dv, dtype=c.f32)
    fwd, bwd, d = c.plan("fwd"), c.plan("bwd"), c.grads()
    saved = bwd.allocate_saved()
    fwd.forward(*c.ins(), y, starts=c.starts, h_in=h_in, h_out=h, slots=sl, saved=saved)
    bwd.backward(*c.ins(), c.dy, saved, **d, starts=c.starts, dh_out=dh_out, dh_in=dh, slots=sl)
    c.check_states("h", h, ref["h"], at, FORWARD)
    c.check_states("dh_in", dh, ref["dh_in"], at, BACKWARD)
    heads = dict(dq=Hk, dk=Hk, dv=Hv, dg=Hv, dbeta=Hv)
    for name in ("dg", "dbeta") if bf16 else heads:
        R.check_heads(name, host(d[name]), ref[name], heads[name], False, BACKWARD, ref.get("mag_" + name))
    if not bf16:
        R.check_heads("y", host(y), ref["y"], Hv, False, FORWARD)
    fwd.check()
    c.b.check_guards()
