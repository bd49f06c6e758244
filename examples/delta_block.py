"""A token-mixing block of a convolutional network, built from the library's calls: a channels-last feature map, a
stream of frames after it, and a training step's gradients.

    normed  = silu(group norm(x))                                  seq_gnorm (over every sample's pixels)
    q, k, v = silu(causal convolution(projection(normed)))         1x1 convolution, seq_conv
    g       = -rate softplus(projection + bias), beta = sigmoid(projection)
    o       = delta rule(q, k, v, g, beta)                         seq_delta (q and k of length 1)
    o       = norm(o) * silu(projection(normed)), a head at a time seq_norm
    out     = x + projection(o)                                    1x1 convolution

The pixels of a sample, in order, are the tokens of a sequence; the states it leaves serve the frames that follow,
a token at a time.  Dense projections are 1x1 convolutions (conv1d with one tap).

    python examples/delta_block.py [--batch 4] [--size 28] [--width 256] [--steps 8]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from convolution_forward_implicit_gb300 import delta, gnorm, seq  # noqa: E402
from convolution_forward_implicit_gb300.binding import CONV_BF16, CONV_EPI_NONE, ConvPlan  # noqa: E402

BF = torch.bfloat16


class Projection:
    """y = x w^T for rows of channels, as a 1x1 convolution.  One plan per number of rows."""

    def __init__(self, w):
        self.w, self.plans = w, {}

    def __call__(self, x):
        k, c = self.w.shape
        rows = x.shape[0]
        if rows not in self.plans:
            p = ConvPlan(1, 1, 1, c, k, (rows,), (1,), (1,), (0,), (1,), CONV_BF16, CONV_EPI_NONE).allocate(x.device)
            p.prepack(self.w)
            self.plans[rows] = p
        y = torch.empty(rows, k, dtype=x.dtype, device=x.device)
        return self.plans[rows].forward(x.contiguous(), None, y)


class DeltaBlock:
    """One block's weights (random, seeded) and its plans by shape."""

    def __init__(self, width, key_heads=2, value_heads=4, head=64, groups=32, taps=4, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        n = lambda *s, std=1.0: torch.randn(*s, generator=gen, device=device) * std      # noqa: E731
        self.width, self.Hk, self.Hv, self.head, self.groups, self.taps = width, key_heads, value_heads, head, groups, taps
        self.K, self.V = key_heads * head, value_heads * head
        self.mixed = 2 * self.K + self.V                       # q, k and v
        self.gn_w, self.gn_b = torch.ones(width, dtype=BF, device=device), n(width, std=0.1).to(BF)
        # q, k, v, then the gate, then g and beta (16 columns at least)
        self.small = max(16, 2 * value_heads)
        self.in_proj = Projection(n(self.mixed + self.V + self.small, width, std=width ** -0.5).to(BF))
        self.conv_w, self.conv_b = n(self.mixed, taps, std=taps ** -0.5).to(BF), n(self.mixed, std=0.1).to(BF)
        self.rate = 1 + 15 * torch.rand(value_heads, generator=gen, device=device)
        step = torch.exp(torch.rand(value_heads, generator=gen, device=device) * math.log(100) + math.log(1e-3))
        self.dt_bias = step + torch.log(-torch.expm1(-step))
        self.head_w = torch.ones(head, dtype=BF, device=device)
        self.out_proj = Projection(n(width, self.V, std=self.V ** -0.5).to(BF))
        self._plans = {}

    def _plan(self, kind, *args, **kw):
        key = (kind, args, tuple(sorted(kw.items())))
        if key not in self._plans:
            self._plans[key] = kind(*args, **kw).allocate()
        return self._plans[key]

    def new_states(self, batch):
        """The states of `batch` sequences at their beginning."""
        dev = self.conv_w.device
        return (torch.zeros(batch, self.taps - 1, self.mixed, dtype=BF, device=dev),
                torch.zeros(batch, self.Hv, self.head, self.head, device=dev))

    def normed(self, x, batch, stats=None):
        y = torch.empty_like(x)
        return self._plan(gnorm.SeqGroupNormPlan, batch, x.shape[0], self.width, self.groups, CONV_BF16, act="silu").forward(
            x, y, w=self.gn_w, b=self.gn_b, stats=stats)

    def decay(self, small):
        """g and beta (fp32) from their projections."""
        H = self.Hv
        return (-self.rate * torch.nn.functional.softplus(small[:, :H].float() + self.dt_bias),
                torch.sigmoid(small[:, H:2 * H].float()))

    def split(self, qkv):
        return qkv[:, :self.K], qkv[:, self.K:2 * self.K], qkv[:, 2 * self.K:]

    def mix(self, normed, batch, states):
        """The tokens of `normed`, (batch L, width), mixed; moves the states on (one token each: a decoding step)."""
        T = normed.shape[0]
        e = lambda *s: torch.empty(*s, dtype=BF, device=normed.device)      # noqa: E731
        conv_state, h = states
        p = self.in_proj(normed)
        raw, gate, small = p[:, :self.mixed], p[:, self.mixed:self.mixed + self.V], p[:, self.mixed + self.V:]
        qkv, o = e(T, self.mixed), e(T, self.V)
        g, beta = self.decay(small)
        heads = (self.Hk, self.Hv, self.head, self.head, CONV_BF16)
        if T == batch:
            self._plan(seq.SeqConvPlan, batch, T, self.mixed, self.taps, CONV_BF16, "step").step(
                raw, self.conv_w, self.conv_b, conv_state, conv_state, qkv)
            self._plan(delta.SeqDeltaPlan, batch, T, *heads, "step").step(*self.split(qkv), g, beta, h, h, o)
        else:
            self._plan(seq.SeqConvPlan, batch, T, self.mixed, self.taps, CONV_BF16).forward(
                raw, self.conv_w, self.conv_b, qkv, state_in=conv_state, state_out=conv_state)
            self._plan(delta.SeqDeltaPlan, batch, T, *heads).forward(*self.split(qkv), g, beta, o, h_in=h, h_out=h)
        rows = T * self.Hv
        out = e(rows, self.head)
        self._plan(seq.SeqNormPlan, rows, self.head, CONV_BF16, post=True, pre=False, residual=False, gate=seq.SEQ_GATE_AFTER).forward(
            o.view(rows, self.head), y=out, gate=gate.contiguous().view(rows, self.head), w_post=self.head_w)
        return self.out_proj(out.view(T, self.V))

    def __call__(self, x, batch, states):
        """x: a feature map (batch, ..., width) bf16; its pixels in order are the tokens."""
        flat = x.reshape(-1, self.width)
        return (flat + self.mix(self.normed(flat, batch), batch, states)).view_as(x)

    def gradients(self, x, qkv, g, beta, do, dnormed, batch):
        """A training step's group norm and delta rule: gradients at q, k, v, g and beta for the gradient do at its output,
        and at the feature map x and the norm's parameters for dnormed."""
        T = qkv.shape[0]
        e = lambda *s, dtype=BF: torch.empty(*s, dtype=dtype, device=x.device)      # noqa: E731
        f32, heads = torch.float32, (self.Hk, self.Hv, self.head, self.head, CONV_BF16)
        fwd, bwd = (self._plan(delta.SeqDeltaPlan, batch, T, *heads, d) for d in ("fwd", "bwd"))
        o, dqkv, saved = e(T, self.V), e(T, self.mixed), bwd.allocate_saved(x.device)
        fwd.forward(*self.split(qkv), g, beta, o, saved=saved)
        dg, dbeta = e(T, self.Hv, dtype=f32), e(T, self.Hv, dtype=f32)
        bwd.backward(*self.split(qkv), g, beta, do, saved, *self.split(dqkv), dg, dbeta)
        stats = e(batch, self.groups, 2, dtype=f32)
        self.normed(x, batch, stats)
        dx, dw, db = e(T, self.width), e(self.width, dtype=f32), e(self.width, dtype=f32)
        self._plan(gnorm.SeqGroupNormPlan, batch, T, self.width, self.groups, CONV_BF16, "bwd", act="silu").backward(
            x, stats, dnormed, dx, w=self.gn_w, b=self.gn_b, dw=dw, db=db)
        return dict(o=o, dqkv=dqkv, dg=dg, dbeta=dbeta, dx=dx, dw=dw, db=db)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--size", type=int, default=28, help="the feature map's height and width")
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args(argv)
    B, L, C, K = a.batch, a.size * a.size, a.width, a.steps
    block = DeltaBlock(C)
    gen = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(BF)      # noqa: E731
    x = n(B, a.size, a.size, C)
    y = block(x, B, block.new_states(B))
    print(f"feature map {tuple(x.shape)} -> {tuple(y.shape)}")

    # the mixer over L tokens and K steps after them, against all at once
    tokens = block.normed(n(B * (L + K), C), B).view(B, L + K, C)
    whole = block.mix(tokens.reshape(-1, C), B, block.new_states(B)).view(B, L + K, C)
    states = block.new_states(B)
    parts = [block.mix(tokens[:, :L].reshape(-1, C).contiguous(), B, states).view(B, L, C)]
    parts += [block.mix(tokens[:, L + i].contiguous(), B, states).view(B, 1, C) for i in range(K)]
    off = (torch.cat(parts, 1).float() - whole.float()).norm() / whole.float().norm()
    print(f"{L} tokens, then {K} steps, against all {L + K} at once: relative difference {off.item():.2e}")

    T = B * L
    g, beta = block.decay(n(T, block.small))
    grads = block.gradients(x.view(T, C), n(T, block.mixed), g, beta, n(T, block.V), n(T, C), B)
    print("gradients: " + ", ".join(f"{k} {tuple(v.shape)}" for k, v in grads.items()))
    return off.item()


if __name__ == "__main__":
    # bf16 activations between the calls: the two ways round alike except where a sum runs in another order for
    # another number of rows
    sys.exit(0 if main() < 1e-2 else 1)
