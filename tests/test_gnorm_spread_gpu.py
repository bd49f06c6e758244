"""The group norm where means differ much within a group: one channel, or one stretch of tokens, far from all others.  Its
variance is a sum of positive terms and keeps its relative accuracy."""
import numpy as np
import pytest

from convolution_forward_implicit_gb300 import gnorm as N
from tests.test_gnorm_gpu import CODE
from tests.test_seq_gpu import Box, host, starts_of

pytestmark = pytest.mark.gpu


def statistics(bf16, b, x, lens, G, ragged=False):
    import torch
    S, (T, D) = len(lens), x.shape
    plan = N.SeqGroupNormPlan(S, T, D, G, CODE[bf16], ragged=ragged, eps=0.0)
    stats, y = b.out(S, G, 2, dtype=torch.float32), b.out(T, D)
    plan.forward(x, y, stats=stats, starts=starts_of(lens) if ragged else None)
    return host(stats), host(y)


def exact(xe, lens, G):
    at, mean, rstd = 0, [], []
    for n in lens:
        x = xe[at:at + n].reshape(n, G, -1)
        mean.append(x.mean((0, 2)))
        rstd.append(1 / np.sqrt(((x - mean[-1][:, None]) ** 2).mean((0, 2))))
        at += n
    return np.array(mean), np.array(rstd)


def check(stats, mean, rstd, terms):
    """terms: additions on the longest way to a variance, each off by half a step (2^-24) of a sum that only grows; rstd takes half of
    its relative error.  The mean's own error goes with the spread, which the sums are taken about."""
    assert (np.abs(stats[..., 1] / rstd - 1) <= 0.5 * (terms + 16) * 2.0 ** -24).all(), np.abs(stats[..., 1] / rstd - 1).max()
    assert (np.abs(stats[..., 0] - mean) <= terms * 2.0 ** -24 * (np.abs(mean) + 1 / rstd)).all()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("D,G,T", [(4096, 1, 700), (2048, 1, 1024), (4096, 1, 1), (1030, 1, 900), (96, 3, 1500), (24, 1, 64)])
@pytest.mark.parametrize("off", [10.0, 100.0, 10000.0])
def test_one_channel_far_from_the_others(bf16, D, G, T, off):
    b = Box(D + T, bf16)
    a = b.rng.standard_normal((T, D))
    a[:, ::D // G] += off
    x, xe = b.put(a)
    mean, rstd = exact(xe, [T], G)
    check(statistics(bf16, b, x, [T], G)[0], mean, rstd, T + D // G)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("D,G,T", [(32, 4, 90000), (1280, 1280, 12000), (64, 64, 700)])
@pytest.mark.parametrize("off", [3.0, 100.0])
def test_a_silent_beginning(bf16, D, G, T, off):
    """The first tokens are zero, all others about `off`."""
    b = Box(D + T, bf16)
    a = b.rng.standard_normal((T, D)) + off
    a[:40] = 0
    x, xe = b.put(a)
    mean, rstd = exact(xe, [T], G)
    check(statistics(bf16, b, x, [T], G)[0], mean, rstd, min(T, 4096))


def test_one_long_sequence_among_many_short_ones():
    b = Box(9, False)
    lens = [3] * 150 + [70000] + [1, 0, 5] * 50
    T, D, G = sum(lens), 64, 8
    x, xe = b.put(b.rng.standard_normal((T, D)) + b.rng.standard_normal(D))
    stats, y = statistics(False, b, x, lens, G, ragged=True)
    live = [i for i, n in enumerate(lens) if n > 0]
    mean, rstd = exact(xe, [n for n in lens if n], G)
    assert (stats[[i for i, n in enumerate(lens) if n == 0]] == 0).all()
    check(stats[live], mean, rstd, 4096)
    i = sum(lens[:150])
    z = ((xe[i:i + 70000].reshape(70000, G, -1) - mean[150][:, None]) * rstd[150][:, None]).reshape(70000, D)
    assert np.abs(y[i:i + 70000] - z).max() <= 1e-4
    b.check_guards()
