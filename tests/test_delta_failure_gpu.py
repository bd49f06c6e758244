"""Failure detection of the delta rule's tensor-core kernels on the GPU without a fault: with the test hook some products are never issued.  The bounded
waits for them run out (about a second), the kernels raise the device error word, see what they issued done, give their tensor memory back and end;
seq_delta_check reports CONV_ERR_TIMEOUT, and the next calls on the same context give what they gave before."""
import os
import time

import pytest

from convolution_forward_implicit_gb300 import binding as B
from convolution_forward_implicit_gb300 import seq as Q
from tests.test_delta_gpu import Case

pytestmark = pytest.mark.gpu


def stalled(c, direction):
    old = os.environ.get("CONV_TEST_STALL")
    os.environ["CONV_TEST_STALL"] = "1"
    try:
        return c.plan(direction).allocate()
    finally:
        if old is None:
            del os.environ["CONV_TEST_STALL"]
        else:
            os.environ["CONV_TEST_STALL"] = old


@pytest.mark.parametrize("Dk", [128, 64])
@pytest.mark.parametrize("L,direction", [(300, "fwd"), (1400, "fwd"), (200, "bwd")])
def test_waits_run_out_and_the_context_recovers(L, direction, Dk):
    import torch
    c = Case(L + Dk, True, [L], 1, 1, Dk, 128, False, decay=0.02)
    fwd, bwd = c.plan("fwd").allocate(), c.plan("bwd").allocate()
    assert (int(Q.seq_plan_describe(fwd.handle).split("piece_chunks=")[1]) > 0) == (L == 1400)
    h, y, d, saved = c.b.out(1, 1, Dk, 128, dtype=c.f32), c.b.out(L, 128), c.grads(), bwd.allocate_saved()

    def run(f, b):
        f.forward(*c.ins(), y, h_out=h, saved=saved)
        b.backward(*c.ins(), c.dy, saved, **d)
        return [t.clone() for t in (y, h, *d.values())]

    want = run(fwd, bwd)
    fwd.check()
    bad = stalled(c, direction)
    torch.cuda.synchronize()
    t0 = time.time()
    if direction == "fwd":
        bad.forward(*c.ins(), y, h_out=h, saved=saved)
    else:
        bad.backward(*c.ins(), c.dy, saved, **d)
    with pytest.raises(B.ConvError) as e:
        bad.check()
    assert e.value.status == B.CONV_ERR_TIMEOUT
    assert 0.8 <= time.time() - t0 <= 30          # it waited out its limit, and ended
    bad.check()                                   # the error word was read and cleared
    again = run(fwd, bwd)
    fwd.check()
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    c.b.check_guards()
