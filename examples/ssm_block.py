"""A selective state space block built from the library's calls: a prompt, decoding token by token, and a
training step's gradients.

    residual, normed = norm(residual + block)                     seq_norm (residual and pre-norm)
    x, z             = in-projection(normed)                      1x1 convolution
    x                = silu(causal convolution(x))                seq_conv
    dt_low, B, C     = projection(x);  dt = projection(dt_low)    1x1 convolutions
    y                = scan(x, dt, A, B, C, D) * silu(z)          seq_scan
    block            = out-projection(y)                          1x1 convolution

Dense projections are 1x1 convolutions (conv1d with one tap), so all arithmetic runs in the library.  They
take whole rows: the columns of dt_low, a slice of x's projection, are copied before theirs.

    python examples/ssm_block.py [--batch 4] [--length 512] [--width 384] [--steps 16]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from convolution_forward_implicit_gb300 import seq  # noqa: E402
from convolution_forward_implicit_gb300.binding import CONV_BF16, CONV_EPI_NONE, ConvPlan  # noqa: E402


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


class SsmBlock:
    """One block's weights (random, seeded) and its plans by shape."""

    def __init__(self, width, states=16, taps=4, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        n = lambda *s, std=1.0: torch.randn(*s, generator=g, device=device) * std      # noqa: E731
        bf = torch.bfloat16
        self.width, self.inner, self.states, self.taps = width, 2 * width, states, taps
        self.rank = max(8, width // 16 // 8 * 8)
        E, R, N = self.inner, self.rank, states
        self.norm_w = torch.ones(width, dtype=bf, device=device)
        self.in_proj = Projection(n(2 * E, width, std=width ** -0.5).to(bf))
        self.conv_w = n(E, taps, std=taps ** -0.5).to(bf)
        self.conv_b = n(E, std=0.1).to(bf)
        self.x_proj = Projection(n(R + 2 * N, E, std=E ** -0.5).to(bf))
        self.dt_proj = Projection(n(E, R, std=R ** -0.5).to(bf))
        step = torch.exp(torch.rand(E, generator=g, device=device) * math.log(100) + math.log(1e-3))
        self.dt_bias = step + torch.log(-torch.expm1(-step))
        self.A = -torch.arange(1, N + 1, device=device).float().repeat(E, 1)
        self.D = torch.ones(E, device=device)
        self.out_proj = Projection(n(width, E, std=E ** -0.5).to(bf))
        self._plans = {}

    def _plan(self, kind, *args, **kw):
        key = (kind, args, tuple(sorted(kw.items())))
        if key not in self._plans:
            self._plans[key] = kind(*args, **kw).allocate()
        return self._plans[key]

    def new_states(self, batch):
        """The states of `batch` sequences at their beginning."""
        dev = self.conv_w.device
        return (torch.zeros(batch, self.taps - 1, self.inner, dtype=torch.bfloat16, device=dev),
                torch.zeros(batch, self.inner, self.states, device=dev))

    def __call__(self, block, residual, batch, states):
        """block: the previous block's output, (batch L, width) bf16; residual: the same, fp32, updated in
        place.  Moves the states on by the L tokens of each sequence; one token each is a decoding step."""
        T, E, N, R = block.shape[0], self.inner, self.states, self.rank
        e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=block.device)      # noqa: E731
        conv_state, h = states
        normed = e(T, self.width)
        self._plan(seq.SeqNormPlan, T, self.width, CONV_BF16).forward(block, y=normed, res=residual, res_out=residual,
                                                                      w_pre=self.norm_w)
        xz = self.in_proj(normed)
        x, z, y = e(T, E), xz[:, E:], e(T, E)
        if T == batch:
            self._plan(seq.SeqConvPlan, batch, T, E, self.taps, CONV_BF16, "step").step(
                xz[:, :E], self.conv_w, self.conv_b, conv_state, conv_state, x)
        else:
            self._plan(seq.SeqConvPlan, batch, T, E, self.taps, CONV_BF16).forward(
                xz[:, :E], self.conv_w, self.conv_b, x, state_in=conv_state, state_out=conv_state)
        dbc = self.x_proj(x)
        args = (x, self.dt_proj(dbc[:, :R]), self.A, dbc[:, R:R + N], dbc[:, R + N:])
        kw = dict(D=self.D, z=z, dt_bias=self.dt_bias)
        if T == batch:
            self._plan(seq.SeqScanPlan, batch, T, E, N, CONV_BF16, "step").step(*args, h, h, y, **kw)
        else:
            self._plan(seq.SeqScanPlan, batch, T, E, N, CONV_BF16).forward(*args, y, h_in=h, h_out=h, **kw)
        return self.out_proj(y)

    def mixer_gradients(self, xz, dt, B, C, dy, batch):
        """A training step's convolution and scan: their gradients at the in-projection's output xz, at dt,
        B and C, and at the parameters, for the gradient dy at the scan's output."""
        T, E, N = xz.shape[0], self.inner, self.states
        e = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device=xz.device)      # noqa: E731
        f32 = torch.float32
        x, y = e(T, E), e(T, E)
        self._plan(seq.SeqConvPlan, batch, T, E, self.taps, CONV_BF16).forward(xz[:, :E], self.conv_w, self.conv_b, x)
        fwd, bwd = (self._plan(seq.SeqScanPlan, batch, T, E, N, CONV_BF16, d) for d in ("fwd", "bwd"))
        saved = bwd.allocate_saved(xz.device)
        kw = dict(D=self.D, z=xz[:, E:], dt_bias=self.dt_bias)
        fwd.forward(x, dt, self.A, B, C, y, saved=saved, **kw)
        g = dict(dx=e(T, E), ddt=e(T, E), dA=e(E, N, dtype=f32), dB=e(T, N), dC=e(T, N))
        more = dict(dD=e(E, dtype=f32), ddt_bias=e(E, dtype=f32))
        dxz = e(T, 2 * E)
        bwd.backward(x, dt, self.A, B, C, dy, saved, **g, dz=dxz[:, E:], **more, **kw)
        dw, db = e(E, self.taps, dtype=f32), e(E, dtype=f32)
        self._plan(seq.SeqConvPlan, batch, T, E, self.taps, CONV_BF16, "bwd").backward(
            xz[:, :E], self.conv_w, self.conv_b, g["dx"], dxz[:, :E], dw, db)
        return dict(y=y, dxz=dxz, dconv_w=dw, dconv_b=db, **{k: g[k] for k in ("ddt", "dA", "dB", "dC")}, **more)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--length", type=int, default=512)
    ap.add_argument("--width", type=int, default=384)
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args(argv)
    B, L, D, K = a.batch, a.length, a.width, a.steps
    block = SsmBlock(D)
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens = torch.randn(B, L + K, D, generator=g, device="cuda").to(torch.bfloat16)

    def run(x, states):
        flat = x.reshape(-1, D).contiguous()
        return block(flat, torch.zeros(flat.shape, device="cuda"), B, states).reshape(B, -1, D)

    whole = run(tokens, block.new_states(B))
    states = block.new_states(B)
    parts = [run(tokens[:, :L], states)]
    parts += [run(tokens[:, L + i:L + i + 1], states) for i in range(K)]
    off = (torch.cat(parts, 1).float() - whole.float()).norm() / whole.float().norm()
    print(f"prompt of {L} tokens, then {K} steps, against all {L + K} at once: relative difference {off.item():.2e}")

    T, E, N = B * L, block.inner, block.states
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)      # noqa: E731
    grads = block.mixer_gradients(n(T, 2 * E), n(T, E), n(T, N), n(T, N), n(T, E), B)
    print("gradients: " + ", ".join(f"{k} {tuple(v.shape)}" for k, v in grads.items()))
    return off.item()


if __name__ == "__main__":
    # bf16 activations between the calls: the two ways round alike except where a projection's sums run in
    # another order for another number of rows
    sys.exit(0 if main() < 1e-2 else 1)
