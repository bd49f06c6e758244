"""The decay's gradient where decay is strong: dg of a token is as small as its factor exp(g), and so are the terms that make it."""
import pytest

from tests import delta_oracle as R
from tests.test_delta_gpu import Case
from tests.test_seq_gpu import host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("Hk,Hv,Dk,Dv", [(1, 2, 128, 128), (2, 2, 64, 64), (1, 1, 48, 80), (1, 3, 128, 36)])
@pytest.mark.parametrize("rate", [5.0, 8.0, 12.0, 16.0])
def test_gradients_of_strong_decay(bf16, Hk, Hv, Dk, Dv, rate):
    """dg_t = <gradient at h'_t, h'_t>; its error goes with the sizes of these products' terms (mag_dg), whatever the outputs' are."""
    c = Case(int(rate) + Dk, bf16, [200, 1, 70, 64], Hk, Hv, Dk, Dv, True, decay=0.1)
    c.g.sub_(rate)
    c.exact["g"] = host(c.g)
    h_in, h0, _, sl = c.states()
    ref = R.delta(**c.exact, lens=c.lens, h0=h0, norm=True, dy=c.dye.reshape(c.T, Hv, Dv))
    y, d, bwd = c.b.out(c.T, Hv * Dv), c.grads(), c.plan("bwd")
    saved = bwd.allocate_saved()
    c.plan("fwd").forward(*c.ins(), y, starts=c.starts, h_in=h_in, slots=sl, saved=saved)
    bwd.backward(*c.ins(), c.dy, saved, **d, starts=c.starts, slots=sl)
    c.check(dict(y=y, **d), ref)
    c.b.check_guards()
