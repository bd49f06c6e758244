"""The gated delta rule on the GPU against the 64-bit oracle (tests/delta_oracle.py): head layouts, sequence lengths, strides and
states where it can go wrong, both types, every direction."""
import numpy as np
import pytest

from convolution_forward_implicit_gb300 import delta as D
from convolution_forward_implicit_gb300 import seq as Q
from convolution_forward_implicit_gb300.binding import CONV_BF16, CONV_F32
from tests import delta_oracle as R
from tests.test_seq_gpu import Box, SENTINEL, host, slots_of, starts_of

pytestmark = pytest.mark.gpu
CODE = {False: CONV_F32, True: CONV_BF16}


class Case:
    """Inputs of one problem on the GPU and their exact values."""

    def __init__(self, seed, bf16, lens, Hk, Hv, Dk, Dv, ragged, norm=True, pad=0, shift=0, decay=0.2, alike=False):
        import torch
        self.b = b = Box(seed, bf16)
        self.bf16, self.lens, self.S, self.T = bf16, lens, len(lens), sum(lens)
        self.Hk, self.Hv, self.Dk, self.Dv, self.norm, self.ragged = Hk, Hv, Dk, Dv, norm, ragged
        T, r = self.T, b.rng

        def keys():
            x = r.standard_normal((T, Hk, Dk))
            if alike:
                x[:] = x[:1]
            return x if norm else x / np.sqrt((x * x).sum(-1, keepdims=True) + 1e-6)

        self.q, qe = b.put(keys().reshape(T, Hk * Dk), pad=pad, shift=shift)
        self.k, ke = b.put(keys().reshape(T, Hk * Dk), pad=pad, shift=shift)
        self.v, ve = b.normal(T, Hv * Dv, pad=pad, shift=shift)
        self.g, ge = b.put(-r.uniform(0, decay, (T, Hv)), dtype=torch.float32, pad=pad)
        self.beta, be = b.put(r.uniform(0, 1, (T, Hv)) if not alike else np.ones((T, Hv)), dtype=torch.float32, pad=pad)
        self.dy, self.dye = b.normal(T, Hv * Dv, pad=pad, shift=shift)
        self.exact = dict(q=qe.reshape(T, Hk, Dk), k=ke.reshape(T, Hk, Dk), v=ve.reshape(T, Hv, Dv), g=ge, beta=be)
        self.starts = starts_of(lens) if ragged else None
        self.pad, self.f32 = pad, torch.float32
        self.kw = dict(ragged=ragged, qk_norm=norm)

    def plan(self, direction, S=None, T=None, **kw):
        return D.SeqDeltaPlan(self.S if S is None else S, self.T if T is None else T, self.Hk, self.Hv, self.Dk, self.Dv, CODE[self.bf16],
                              direction, **{**self.kw, **kw})

    def ins(self):
        return self.q, self.k, self.v, self.g, self.beta

    def grads(self):
        o = self.b.out
        K, V, H, T = self.Hk * self.Dk, self.Hv * self.Dv, self.Hv, self.T
        return dict(dq=o(T, K, pad=self.pad), dk=o(T, K, pad=self.pad), dv=o(T, V, pad=self.pad), dg=o(T, H, dtype=self.f32, pad=self.pad),
                    dbeta=o(T, H, dtype=self.f32, pad=self.pad))

    def states(self, drop=(), std=0.3):
        """State rows in any order, some sequences without one: the buffer, their exact values by sequence, slots."""
        at, sl = slots_of(self.S, self.b.rng, self.S + 2, drop)
        buf, full = self.b.normal(self.S + 2, self.Hv, self.Dk, self.Dv, std=std, dtype=self.f32)
        return buf, np.where((at >= 0)[:, None, None, None], full[at], 0), at, sl

    def check(self, got, ref):
        T, heads = self.T, dict(y=self.Hv, dq=self.Hk, dk=self.Hk, dv=self.Hv, dg=self.Hv, dbeta=self.Hv)
        for name, t in got.items():
            low = self.bf16 and name in ("y", "dq", "dk", "dv")
            R.check_heads(name, host(t), ref[name], heads[name], low, R.FORWARD if name == "y" else R.BACKWARD, ref.get("mag_" + name))

    def check_states(self, name, buf, ref, at, tol):
        got, named = host(buf), set(at[at >= 0])
        for s in range(self.S):
            if at[s] >= 0:
                for h in range(self.Hv):
                    R.check(f"{name} of sequence {s} head {h}", got[at[s], h], ref[s, h], False, tol)
        for r in range(self.S + 2):
            if r not in named:
                assert (got[r] == SENTINEL).all()


UNIFORM = [[1], [64], [65], [7] * 3, [200], [1] * 5]
RAGGED = [[0, 1, 0, 0, 5, 2, 0], [3, 140, 1, 17], [0], [64, 0, 64, 1], [129, 3, 63, 128]]
HEADS = [(1, 1, 128, 128), (2, 4, 64, 64), (1, 3, 37, 19), (2, 2, 16, 8), (1, 2, 104, 200), (1, 1, 1, 1), (3, 3, 128, 16), (1, 2, 72, 24)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("lens,ragged", [(v, False) for v in UNIFORM] + [(v, True) for v in RAGGED])
@pytest.mark.parametrize("Hk,Hv,Dk,Dv", HEADS)
def test_delta(bf16, lens, ragged, Hk, Hv, Dk, Dv):
    """Outputs, states left and every gradient, states in any slots."""
    norm, pad = (Dk + len(lens)) % 2 == 0, [0, 8, 3][(Dv + sum(lens)) % 3]
    c = Case(7 * Dk + Dv + sum(lens), bf16, lens, Hk, Hv, Dk, Dv, ragged, norm=norm, pad=pad)
    drop = [c.S // 2] if c.S > 2 else []
    h_in, h0, at, sl = c.states(drop)
    dh_out, _ = c.b.normal(c.S + 2, Hv, Dk, Dv, dtype=c.f32)
    dhe = np.where((at >= 0)[:, None, None, None], host(dh_out)[at], 0)
    ref = R.delta(**c.exact, lens=lens, h0=h0, norm=norm, dy=c.dye.reshape(c.T, Hv, Dv), dh_out=dhe)
    y, h_out = c.b.out(c.T, Hv * Dv, pad=pad), c.b.out(c.S + 2, Hv, Dk, Dv, dtype=c.f32)
    bwd = c.plan("bwd")
    saved = bwd.allocate_saved()
    saved.fill_(float("nan"))
    fwd = c.plan("fwd").allocate()
    if fwd.workspace is not None:
        fwd.workspace.fill_(0xFF)                   # (NaN in every type)
    fwd.forward(*c.ins(), y, starts=c.starts, h_in=h_in, h_out=h_out, slots=sl, saved=saved)
    c.check(dict(y=y), ref)
    c.check_states("h", h_out, ref["h"], at, R.FORWARD)
    bwd.allocate()
    if bwd.workspace is not None:
        bwd.workspace.fill_(0xFF)
    d, dh_in = c.grads(), c.b.out(c.S + 2, Hv, Dk, Dv, dtype=c.f32)
    bwd.backward(*c.ins(), c.dy, saved, **d, starts=c.starts, dh_out=dh_out, dh_in=dh_in, slots=sl)
    c.check(d, ref)
    c.check_states("dh_in", dh_in, ref["dh_in"], at, R.BACKWARD)
    fwd.check()
    c.b.check_guards()
    # the same bits again, in place of the states, without saving
    both, y2 = h_in.clone(), c.b.out(c.T, Hv * Dv, pad=pad)
    fwd.forward(*c.ins(), y2, starts=c.starts, h_in=both, h_out=both, slots=sl)
    assert bool((y2 == y).all())
    left = host(both)
    for s in range(c.S):
        if at[s] >= 0:
            assert np.array_equal(left[at[s]], host(h_out)[at[s]])
    d2 = c.grads()
    bwd.backward(*c.ins(), c.dy, saved, **d2, starts=c.starts, dh_out=dh_out, slots=sl)
    for k in d:
        assert bool((d[k] == d2[k]).all()), k


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("S,Hk,Hv,Dk,Dv", [(1, 1, 1, 128, 128), (3, 2, 4, 64, 64), (5, 1, 3, 37, 19), (2, 1, 1, 1, 1), (70, 1, 2, 16, 36), (2, 2, 2, 128, 260)])
def test_steps_continue_a_prompt(bf16, S, Hk, Hv, Dk, Dv):
    """A prompt and one-token steps, in place and with dropped slots, give what the whole sequence gives."""
    L, more = 70, 3
    c = Case(S + Dk, bf16, [L + more] * S, Hk, Hv, Dk, Dv, False)
    ref = R.delta(**c.exact, lens=c.lens, h0=np.zeros((S, Hv, Dk, Dv)), norm=True)
    three = lambda t: t.reshape(S, L + more, -1)                       # noqa: E731
    ins, want = [three(t) for t in c.ins()], three(ref["y"])
    h = c.b.out(S, Hv, Dk, Dv, dtype=c.f32)
    y = c.b.out(S * L, Hv * Dv)
    c.plan("fwd", T=S * L).forward(*(t[:, :L].contiguous() for t in ins), y, h_out=h)
    R.check_heads("prompt", host(y).reshape(S * L, -1), want[:, :L].reshape(S * L, -1), Hv, bf16, R.FORWARD)
    step = c.plan("step", T=S)
    out = c.b.out(S, Hv * Dv)
    for i in range(more):
        step.step(*(t[:, L + i] for t in ins), h, h, out)
        R.check_heads(f"step {i}", host(out), want[:, L + i], Hv, bf16, R.FORWARD)
    for s in range(S):
        R.check("state", host(h)[s], ref["h"][s], False, R.FORWARD)
    # without states: from zero, nothing left; a dropped slot likewise
    step.step(*(t[:, 0] for t in ins), None, None, out)
    R.check_heads("first", host(out), want[:, 0], Hv, bf16, R.FORWARD)
    if S > 2:
        at, sl = slots_of(S, c.b.rng, S, drop=[1])
        before = h.clone()
        step.step(*(t[:, 0] for t in ins), None, h, out, slots=sl)
        free = sorted(set(range(S)) - set(at[at >= 0]))
        assert bool((h[free] == before[free]).all())
        one = R.delta(**{k: v.reshape(S, L + more, *v.shape[1:])[:, 0] for k, v in c.exact.items()}, lens=[1] * S, h0=np.zeros((S, Hv, Dk, Dv)), norm=True)
        for s in range(S):
            if at[s] >= 0:
                R.check("state", host(h)[at[s]], one["h"][s], False, R.FORWARD)
    c.b.check_guards()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("Dk,Dv,shift", [(32, 32, 1), (128, 128, 1), (64, 64, 4), (33, 7, 1)])
def test_rows_at_any_element(bf16, Dk, Dv, shift):
    """Rows that are not aligned to 16 bytes give what aligned ones give."""
    c = Case(3, bf16, [100, 37], 1, 2, Dk, Dv, True, pad=1, shift=shift)
    ref = R.delta(**c.exact, lens=c.lens, h0=np.zeros((2, 2, Dk, Dv)), norm=True, dy=c.dye.reshape(c.T, 2, Dv))
    y, d, bwd = c.b.out(c.T, 2 * Dv, pad=1), c.grads(), c.plan("bwd")
    saved = bwd.allocate_saved()
    c.plan("fwd").forward(*c.ins(), y, starts=c.starts, saved=saved)
    bwd.backward(*c.ins(), c.dy, saved, **d, starts=c.starts)
    c.check(dict(y=y, **d), ref)
    c.b.check_guards()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("Dk,Dv", [(128, 128), (48, 80)])
def test_tokens_that_drop_the_state(bf16, Dk, Dv):
    """g of minus infinity, or far below what exp can hold, forgets what was before; nothing becomes infinite or NaN."""
    c = Case(11, bf16, [150], 1, 2, Dk, Dv, False, decay=3.0)
    g = c.g.clone()
    at = [0, 1, 30, 63, 64, 100, 149]
    for i, t in enumerate(at):
        g[t] = [-float("inf"), -3.4e38, -250.0][i % 3]
    c.g, c.exact["g"] = g, host(g)
    h_in, h0, _, sl = c.states()
    ref = R.delta(**c.exact, lens=c.lens, h0=h0, norm=True, dy=c.dye.reshape(c.T, 2, Dv))
    y, d, bwd = c.b.out(c.T, 2 * Dv), c.grads(), c.plan("bwd")
    saved = bwd.allocate_saved()
    c.plan("fwd").forward(*c.ins(), y, h_in=h_in, slots=sl, saved=saved)
    bwd.backward(*c.ins(), c.dy, saved, **d)
    c.check(dict(y=y, **d), ref)
    assert bool((d["dg"][at] == 0).all())
    # one token at a time
    h, out, step = h_in[sl.long()].contiguous(), c.b.out(1, 2 * Dv), c.plan("step", T=1)
    for t in range(3):
        step.step(*(x[t:t + 1] for x in c.ins()), h, h, out)
        R.check_heads("step", host(out), ref["y"][t:t + 1], 2, bf16, R.FORWARD)


@pytest.mark.parametrize("bf16", [False, True])
def test_keys_that_are_all_alike(bf16):
    """One key, beta 1 and no decay: every token replaces the value before it (the triangular system is as far from
    the identity as it gets)."""
    c = Case(12, bf16, [190], 1, 1, 64, 64, False, decay=0.0, alike=True)
    ref = R.delta(**c.exact, lens=c.lens, h0=np.zeros((1, 1, 64, 64)), norm=True, dy=c.dye.reshape(190, 1, 64))
    y, h, bwd = c.b.out(190, 64), c.b.out(1, 1, 64, 64, dtype=c.f32), c.plan("bwd")
    saved, d = bwd.allocate_saved(), c.grads()
    c.plan("fwd").forward(*c.ins(), y, h_out=h, saved=saved)
    bwd.backward(*c.ins(), c.dy, saved, **d)
    c.check(dict(y=y, **d), ref)
    R.check("h", host(h)[0, 0], ref["h"][0, 0], False, R.FORWARD)


@pytest.mark.parametrize("bf16", [False, True])
def test_bad_values_stay_in_their_sequence_and_head(bf16):
    import torch
    c = Case(13, bf16, [100, 90, 70], 2, 4, 64, 64, True)
    y0, bwd, fwd = c.b.out(c.T, 256), c.plan("bwd"), c.plan("fwd")
    saved, d0 = bwd.allocate_saved(), c.grads()
    fwd.forward(*c.ins(), y0, starts=c.starts, saved=saved)
    bwd.backward(*c.ins(), c.dy, saved, **d0, starts=c.starts)
    c.v[120, 64:128] = float("nan")                 # sequence 1, value head 1 (key head 0)
    c.v[130, 64] = float("inf")
    y, d = c.b.out(c.T, 256), c.grads()
    fwd.forward(*c.ins(), y, starts=c.starts, saved=saved)
    bwd.backward(*c.ins(), c.dy, saved, **d, starts=c.starts)
    for name, new, old in [("y", y, y0)] + [(k, d[k], d0[k]) for k in d]:
        heads = 2 if name in ("dq", "dk") else 4
        a, b = new.reshape(c.T, heads, -1), old.reshape(c.T, heads, -1)
        keep = torch.ones(c.T, heads, dtype=torch.bool, device="cuda")
        keep[100:190, 0 if heads == 2 else 1] = False
        assert bool((a[keep] == b[keep]).all()), name
    assert bool(torch.isnan(y[189, 64:128].float()).all())


def test_a_scale_of_its_own():
    c = Case(14, False, [80], 1, 1, 32, 32, False)
    y = c.b.out(80, 32)
    c.plan("fwd", scale=-0.7).forward(*c.ins(), y)
    ref = R.delta(**c.exact, lens=[80], h0=np.zeros((1, 1, 32, 32)), norm=True, scale=-0.7)
    c.check(dict(y=y), ref)


@pytest.mark.parametrize("bf16", [False, True])
def test_rows_beyond_32_bit_offsets(bf16):
    """q, k, v and y as slices of rows so long that the last tokens lie beyond 2^31 elements."""
    import torch
    T, ld, K, V = 600, 1 << 22, 64, 64
    t = torch.bfloat16 if bf16 else torch.float32
    wide = torch.empty((T - 1) * ld + 4 * K, dtype=t, device="cuda")
    assert wide.numel() > 1 << 31
    cut = lambda i: wide.as_strided((T, K), (ld, 1), i * K)             # noqa: E731
    c = Case(15, bf16, [T], 1, 1, K, V, False)
    for i, x in enumerate((c.q, c.k, c.v)):
        cut(i).copy_(x)
    want, got = c.b.out(T, V), cut(3)
    fwd = c.plan("fwd")
    fwd.forward(*c.ins(), want)
    fwd.forward(cut(0), cut(1), cut(2), c.g, c.beta, got)
    assert bool((got == want).all())
    del wide
    torch.cuda.empty_cache()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("S,L,Hk,Hv,Dk,Dv", [(4, 2000, 16, 16, 128, 128), (4, 1000, 8, 32, 128, 128), (6, 700, 12, 12, 64, 192)])
def test_a_large_batch_gives_what_its_sequences_give(bf16, S, L, Hk, Hv, Dk, Dv):
    """Many times more chunks and heads than run at once: the bits of every sequence alone, each time."""
    import torch
    T = S * L
    gen = torch.Generator("cuda").manual_seed(S + L)
    dtype = torch.bfloat16 if bf16 else torch.float32

    def normal(cols, dtype=dtype):
        return torch.randn(T, cols, generator=gen, device="cuda").to(dtype)

    ins = [normal(Hk * Dk), normal(Hk * Dk), normal(Hv * Dv), -0.1 * normal(Hv, torch.float32).abs(), torch.sigmoid(normal(Hv, torch.float32))]
    dy = normal(Hv * Dv)

    def plans(n):
        return (D.SeqDeltaPlan(n, n * L, Hk, Hv, Dk, Dv, CODE[bf16], d, qk_norm=True) for d in ("fwd", "bwd"))

    f, b = plans(S)
    saved, y, chunks = b.allocate_saved(), torch.empty_like(dy), S * (-(-L // 64)) * Hv
    assert saved.numel() == chunks * (Dk + 64) * Dv

    def backward(plan, saved, rows):
        x = [t[rows] for t in ins]
        out = [torch.empty_like(t) for t in x]
        plan.backward(*x, dy[rows], saved, *out)
        return out

    saved.fill_(float("nan"))
    f.forward(*ins, y, saved=saved)
    states, tokens = saved[:chunks * Dk * Dv].view(S, -1), saved[chunks * Dk * Dv:].view(S, -1)
    alone, one = [], torch.empty_like(y[:L])
    fa, ba = plans(1)
    for s in range(S):
        rows = slice(s * L, (s + 1) * L)
        alone.append(backward(ba, torch.cat((states[s], tokens[s])), rows))
        # the walk of one sequence may be cut where the batch's is not: sums of fp32 in another order, and a rounding
        fa.forward(*(t[rows] for t in ins), one)
        close = (2.0 ** -7 if bf16 else 1e-5) * one.float().abs().max()
        assert float((one.float() - y[rows].float()).abs().max()) <= float(close)
    want = [torch.cat(t) for t in zip(*alone)]
    assert all(bool(t.isfinite().all()) for t in (y, *want))
    again = torch.empty_like(y)
    for _ in range(4):
        f.forward(*ins, again, saved=saved)
        assert torch.equal(y, again)
        for name, a, b_ in zip(("dq", "dk", "dv", "dg", "dbeta"), backward(b, saved, slice(None)), want):
            assert torch.equal(a, b_), name
    f.check()


# the last: whether the axis is cut
CUT = [([2000], False, 1, 2, 128, 128, True), ([1500] * 2, False, 1, 2, 64, 64, True), ([700, 0, 1300, 64, 1, 65], True, 1, 1, 104, 200, True),
       ([900, 1, 1100], True, 1, 2, 37, 19, True), ([1290], False, 2, 2, 16, 16, True), ([640, 641], True, 1, 1, 128, 128, False)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("lens,ragged,Hk,Hv,Dk,Dv,cut", CUT)
def test_pieces_of_long_sequences(bf16, lens, ragged, Hk, Hv, Dk, Dv, cut):
    """Few heads and long sequences: the axis is cut for the walk, and what the pieces start from is joined."""
    c = Case(Dk + Dv + len(lens), bf16, lens, Hk, Hv, Dk, Dv, ragged, norm=True, decay=0.02)
    fwd, bwd = c.plan("fwd"), c.plan("bwd")
    assert (int(Q.seq_plan_describe(fwd.handle).split("piece_chunks=")[1]) > 0) == cut
    h_in, h0, at, sl = c.states([1] if c.S > 2 else [])
    ref = R.delta(**c.exact, lens=lens, h0=h0, norm=True, dy=c.dye.reshape(c.T, Hv, Dv))
    fwd.allocate()
    fwd.workspace.fill_(0xFF)
    y, h_out, saved = c.b.out(c.T, Hv * Dv), c.b.out(c.S + 2, Hv, Dk, Dv, dtype=c.f32), bwd.allocate_saved()
    saved.fill_(float("nan"))
    fwd.forward(*c.ins(), y, starts=c.starts, h_in=h_in, h_out=h_out, slots=sl, saved=saved)
    c.check(dict(y=y), ref)
    c.check_states("h", h_out, ref["h"], at, R.FORWARD)
    d = c.grads()
    bwd.backward(*c.ins(), c.dy, saved, **d, starts=c.starts, slots=sl)
    c.check(d, ref)
    fwd.check()
    c.b.check_guards()
    both, y2 = h_in.clone(), c.b.out(c.T, Hv * Dv)
    fwd.forward(*c.ins(), y2, starts=c.starts, h_in=both, h_out=both, slots=sl)
    assert bool((y2 == y).all())
    left, want = host(both), host(h_out)
    for s in range(c.S):
        if at[s] >= 0:
            assert np.array_equal(left[at[s]], want[at[s]])
    # rows that are not whole 16-byte groups, and no state: kernels of their own in bf16
    o = Case(Dk + Dv + len(lens), bf16, lens, Hk, Hv, Dk, Dv, ragged, norm=True, decay=0.02, shift=1)
    ref = R.delta(**o.exact, lens=lens, h0=0 * h0, norm=True)
    fwd.forward(*o.ins(), y2, starts=o.starts)
    o.check(dict(y=y2), ref)


def test_many_sequences():
    """More sequences than a launch's second dimension holds."""
    import torch
    S, T = 70000, 140000
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")            # noqa: E731
    q, k, v = n(T, 8), n(T, 8), n(T, 4)
    gg, beta = -torch.rand(T, 1, generator=g, device="cuda"), torch.rand(T, 1, generator=g, device="cuda")
    starts = torch.arange(0, T + 1, 2, dtype=torch.int32, device="cuda")
    y, y2 = torch.empty(T, 4, device="cuda"), torch.empty(T, 4, device="cuda")
    h, h2 = torch.empty(S, 1, 8, 4, device="cuda"), torch.empty(S, 1, 8, 4, device="cuda")
    D.SeqDeltaPlan(S, T, 1, 1, 8, 4, CONV_F32, ragged=True).forward(q, k, v, gg, beta, y, starts=starts, h_out=h)
    step = D.SeqDeltaPlan(S, S, 1, 1, 8, 4, CONV_F32, "step")
    row = lambda t, i: t.view(S, 2, -1)[:, i]                             # noqa: E731
    step.step(*(row(t, 0) for t in (q, k, v, gg, beta)), None, h2, row(y2, 0))
    step.step(*(row(t, 1) for t in (q, k, v, gg, beta)), h2, h2, row(y2, 1))
    # both forms are within the bound of the definition
    size = float(y.square().mean().sqrt())
    assert float((y - y2).abs().max()) <= 64 * R.FORWARD * size and float((h - h2).square().mean().sqrt()) <= 2 * R.FORWARD * float(h.square().mean().sqrt())


def test_bounds_outside_their_contract():
    """Sequence bounds that are not in order give other results and touch nothing outside the tensors."""
    import torch
    for bf16 in (False, True):
        c = Case(16, bf16, [60, 80, 30], 1, 2, 64, 64, True)
        for bad in ([0, 500, -7, 170], [0, 100, 20, 170], [90, 10, 5, 2], [0, 0, 0, 0]):
            st = torch.tensor(bad, dtype=torch.int32, device="cuda")
            y, d, bwd = c.b.out(c.T, 128), c.grads(), c.plan("bwd")
            saved = bwd.allocate_saved()
            h = c.b.out(3, 2, 64, 64, dtype=c.f32)
            c.plan("fwd").forward(*c.ins(), y, starts=st, h_out=h, saved=saved)
            bwd.backward(*c.ins(), c.dy, saved, **d, starts=st)
            c.b.check_guards()


def test_bounds_outside_their_contract_in_pieces():
    import torch
    for bf16 in (False, True):
        c = Case(22, bf16, [900, 1000, 300], 1, 2, 64, 64, True)
        fwd, bwd = c.plan("fwd"), c.plan("bwd")
        assert int(Q.seq_plan_describe(fwd.handle).split("piece_chunks=")[1]) > 0
        for bad in ([0, 5000, -7, 2200], [0, 2000, 20, 2200], [1900, 10, 5, 2], [0, 0, 0, 0]):
            st = torch.tensor(bad, dtype=torch.int32, device="cuda")
            y, h = c.b.out(c.T, 128), c.b.out(3, 2, 64, 64, dtype=c.f32)
            fwd.forward(*c.ins(), y, starts=st, h_out=h, saved=bwd.allocate_saved())
            c.b.check_guards()


# ------------------------------------------------------------------------------- streams and graphs
def test_streams_and_graphs():
    """A prompt and its backward call on another stream, two streams with one plan, and captured; an eager autograd graph
    of the same tensors lives meanwhile."""
    import torch
    c = Case(17, True, [300], 2, 4, 128, 128, False)
    fwd, bwd = c.plan("fwd"), c.plan("bwd")
    saved, y, d = bwd.allocate_saved(), c.b.out(300, 512), c.grads()
    leaf = c.v.clone().requires_grad_()
    loss = (leaf.float() ** 2).sum()

    def run(**kw):
        fwd.forward(*c.ins(), y, saved=saved, **kw)
        bwd.backward(*c.ins(), c.dy, saved, **d, **kw)

    run()
    torch.cuda.synchronize()
    want = {k: t.clone() for k, t in dict(y=y, **d).items()}

    def same():
        torch.cuda.synchronize()
        for k, t in dict(y=y, **d).items():
            assert torch.equal(t, want[k]), k
            t.fill_(1.0)

    same()
    side = [torch.cuda.Stream() for _ in range(2)]
    for s in side:
        torch.cuda.synchronize()
        run(stream=s.cuda_stream)
        same()
    torch.cuda.synchronize()
    with torch.cuda.stream(side[0]):
        run()
    side[1].wait_stream(side[0])
    with torch.cuda.stream(side[1]):
        run()
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        graph.replay()
        same()
    loss.backward()
    assert torch.equal(leaf.grad, (2 * leaf.detach().float()).to(leaf.dtype))
    fwd.check()


@pytest.mark.parametrize("bf16", [False, True])
def test_pieces_on_streams_and_in_a_graph(bf16):
    """A plan that cuts the axis, in place of its states: on two streams one after the other, and captured and replayed."""
    import torch
    c = Case(23, bf16, [1400], 1, 2, 128, 128, False, decay=0.02)
    fwd, y = c.plan("fwd"), c.b.out(1400, 256)
    assert int(Q.seq_plan_describe(fwd.handle).split("piece_chunks=")[1]) > 0
    h0, _ = c.b.normal(1, 2, 128, 128, std=0.3, dtype=c.f32)
    h = h0.clone()
    fwd.forward(*c.ins(), y, h_in=h, h_out=h)
    want = y.clone(), h.clone()
    side = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for s in side:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                h.copy_(h0)
                y.fill_(1.0)
                fwd.forward(*c.ins(), y, h_in=h, h_out=h)
            torch.cuda.current_stream().wait_stream(s)
            assert torch.equal(y, want[0]) and torch.equal(h, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h.copy_(h0)
        fwd.forward(*c.ins(), y, h_in=h, h_out=h)
    for _ in range(3):
        y.fill_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(h, want[1])
    fwd.check()


def test_two_calls_at_once():
    """Two plans of one problem on two streams, each with its own workspace."""
    import torch
    c = Case(18, True, [500], 2, 2, 128, 128, False)
    plans, outs = [c.plan("fwd") for _ in range(2)], [c.b.out(500, 256) for _ in range(2)]
    side = [torch.cuda.Stream() for _ in range(2)]
    want = c.b.out(500, 256)
    c.plan("fwd").forward(*c.ins(), want)
    torch.cuda.synchronize()
    for _ in range(5):
        for p, y, s in zip(plans, outs, side):
            p.forward(*c.ins(), y, stream=s.cuda_stream)
    torch.cuda.synchronize()
    assert all(bool((y == want).all()) for y in outs)
    assert plans[0].workspace.data_ptr() != plans[1].workspace.data_ptr()


def test_tensors_are_on_the_current_gpu():
    import torch
    from convolution_forward_implicit_gb300.binding import ConvError
    c = Case(19, False, [10], 1, 1, 16, 16, False)
    with pytest.raises(ConvError):
        c.plan("fwd").forward(c.q.cpu(), *c.ins()[1:], c.b.out(10, 16))
    with pytest.raises(ConvError):
        c.plan("fwd").forward(c.q, c.k.cpu(), c.v, c.g, c.beta, c.b.out(10, 16))
    with pytest.raises(ConvError):
        c.plan("fwd").forward(c.q, c.k, c.v, c.g.to(torch.bfloat16), c.beta, c.b.out(10, 16))
    assert Q.seq_plan_describe(c.plan("fwd").handle).startswith("op=delta direction=fwd dtype=f32")


def test_gradients_against_differences():
    """The loss's change along a direction, from two forward calls in fp32, against the gradients' product with it."""
    c = Case(20, False, [90, 40], 1, 2, 32, 24, True)
    y, bwd = c.b.out(c.T, 48), c.plan("bwd")
    saved, d = bwd.allocate_saved(), c.grads()
    fwd = c.plan("fwd")
    fwd.forward(*c.ins(), y, starts=c.starts, saved=saved)
    bwd.backward(*c.ins(), c.dy, saved, **d, starts=c.starts)
    dy = host(c.dy)
    names = ("q", "k", "v", "g", "beta")
    import torch
    for i, name in enumerate(names):
        ins = list(c.ins())
        step = c.b.rng.standard_normal(tuple(ins[i].shape))
        move = torch.from_numpy(step).float().cuda()
        eps, loss = 2.0 ** -8, []
        for sign in (1, -1):
            ins[i] = c.ins()[i] + sign * eps * move
            fwd.forward(*ins, y, starts=c.starts)
            loss.append(float((host(y) * dy).sum()))
        num, ana = (loss[0] - loss[1]) / (2 * eps), float((host(d["d" + name]) * host(move)).sum())
        # the difference's own error: eps^2 of the third derivative, and the rounding of two sums over eps
        size = float(np.linalg.norm(host(d["d" + name])) * np.linalg.norm(step)) / np.sqrt(step.size)
        assert abs(num - ana) <= 0.02 * size + 1e-3 * abs(ana), (name, num, ana, size)


# ---------------------------------------------------------------------------------- together
def test_block_example():
    """examples/delta_block.py: the mixer over a prompt and steps behind it against all tokens at once.  Between the calls every
    activation is rounded to bf16 (2^-9 relative); the two ways differ by such roundings only, over the handful of them
    that a token passes: far below 1e-2."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import delta_block
    assert delta_block.main(["--batch", "2", "--size", "9", "--width", "64", "--steps", "4"]) < 1e-2


def test_block_example_gradients():
    """The example's training step against the 64-bit oracle, on the tensors that it made."""
    import os
    import sys
    import torch
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import delta_block
    B, L, C = 2, 90, 64
    block = delta_block.DeltaBlock(C, head=32)
    b, T = Box(21, True), B * L
    x, xe = b.normal(T, C)
    qkv, qe = b.normal(T, block.mixed)
    do, doe = b.normal(T, block.V)
    dn, dne = b.normal(T, C)
    small, _ = b.normal(T, block.small)
    g, beta = block.decay(small)
    got = block.gradients(x, qkv, g, beta, do, dn, B)
    q, k, v = (host(t) for t in block.split(qkv))
    cut = lambda t, h: t.reshape(T, h, -1)                              # noqa: E731
    ref = R.delta(cut(q, block.Hk), cut(k, block.Hk), cut(v, block.Hv), host(g), host(beta), [L] * B,
                  np.zeros((B, block.Hv, 32, 32)), True, dy=cut(doe, block.Hv))
    R.check_heads("o", host(got["o"]), ref["y"], block.Hv, True, R.FORWARD)
    for name, part, heads in zip(("dq", "dk", "dv"), block.split(got["dqkv"]), (block.Hk, block.Hk, block.Hv)):
        R.check_heads(name, host(part), ref[name], heads, True, R.BACKWARD)
    for name in ("dg", "dbeta"):
        R.check_heads(name, host(got[name]), ref[name], block.Hv, False, R.BACKWARD, ref["mag_" + name])
    ref, mag = R.gnorm(xe, host(block.gn_w), host(block.gn_b), block.groups, [L] * B, "silu", 1e-5, dy=dne)
    for name in ("dx", "dw", "db"):
        R.O.check(name, host(got[name]), ref[name], mag[name], 400 + T, name == "dx")
    assert torch.isfinite(got["dx"].float()).all()
