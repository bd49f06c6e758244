"""Tight bounds of the delta rule's fp32 results on ordinary inputs (keys of length 1 that are not alike, little decay), and that they tell a lost
low part of an operand and a wrong term of each gradient.

An addition of a product in parts cuts at most 2^-23 of its partial sum, half of that in the mean, always towards zero.  48 of them (128 terms in
steps of 8, three products of parts) leave 48 2^-24 = 2.9e-6 of the result.  Forward K h, T R (T's norm below 3 for these keys) and K^T U or A U follow one
another: (1 + 3 + 1) 2.9e-6 = 1.5e-5.  The gradients go through about twice as many: 3e-5.  A lost low part of a tf32 operand is 2^-12 of each value,
rounded to nearest: 7e-5 to 1.4e-4 of the norm."""
import numpy as np
import pytest

from tests import delta_oracle as R

FORWARD, BACKWARD = 1.5e-5, 3e-5


def tf32(x):
    """Rounded to 11 bits."""
    m, e = np.frexp(x)
    return np.ldexp(np.round(m * 2048) / 2048, e)


def inputs(rng, T, H, K, V):
    n = rng.standard_normal
    return dict(q=n((T, H, K)), k=n((T, H, K)), v=n((T, H, V)), g=-rng.uniform(0, 0.05, (T, H)), beta=rng.uniform(0, 1, (T, H)), h0=n((1, H, K, V)) * 0.3)


@pytest.mark.parametrize("lost", ["state", "values", "keys"])
def test_bounds_tell_a_lost_low_part(lost):
    """The state at every chunk's start, every u's value, or the keys, in 11 bits."""
    rng = np.random.default_rng(1)
    T, H, K, V = 192, 2, 64, 48
    a = inputs(rng, T, H, K, V)
    ref = R.delta(**a, lens=[T], norm=True)
    if lost == "state":
        h, ys = a["h0"], []
        for t in range(0, T, 64):
            part = {n: x[t:t + 64] for n, x in a.items() if n != "h0"}
            o = R.delta(**part, h0=tf32(h), lens=[64], norm=True)
            h = o["h"]
            ys.append(o["y"])
        got = dict(y=np.concatenate(ys), h=h)
    else:
        a = dict(a, **{"v" if lost == "values" else "k": tf32(a["v" if lost == "values" else "k"])})
        got = R.delta(**a, lens=[T], norm=True)
    with pytest.raises(AssertionError):
        R.check_heads("y", got["y"], ref["y"], H, False, FORWARD)
    with pytest.raises(AssertionError):
        for h in range(H):
            R.check("h", got["h"][0, h], ref["h"][0, h], False, FORWARD)


@pytest.mark.parametrize("name", ["dq", "dk", "dv", "dg", "dbeta"])
@pytest.mark.parametrize("fault", ["a low part", "one token late", "another's head", "one row"])
def test_bounds_tell_wrong_gradients(name, fault):
    rng = np.random.default_rng(2)
    T, H, K, V = 150, 2, 32, 24
    a = inputs(rng, T, H, K, V)
    ref = R.delta(**a, lens=[T], norm=True, dy=rng.standard_normal((T, H, V)), dh_out=rng.standard_normal((1, H, K, V)))
    wrong = ref[name].reshape(T, H, -1).copy()
    if fault == "a low part":
        terms = ref.get("mag_" + name, np.abs(ref[name])).reshape(wrong.shape)
        wrong = wrong + 2.0 ** -12 * terms * rng.uniform(-1, 1, wrong.shape)
    elif fault == "one token late":
        wrong[64:] = np.roll(wrong[64:], 1, 0)
    elif fault == "another's head":
        wrong = wrong[:, ::-1]
    else:
        wrong[127] *= 1 + 2.0 ** -5
    with pytest.raises(AssertionError):
        R.check_heads(name, wrong.reshape(T, -1), ref[name], H, False, BACKWARD, ref.get("mag_" + name))
