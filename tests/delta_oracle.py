"""The gated delta rule and the group norm with an activation in 64 bits from their formulas (numpy), with gradients.

Bounds of the delta rule.  With keys of length 1, beta in [0, 1] and decay factors of at most 1 every step contracts
(|I - beta k k^T| <= 1), so an error made in one place does not grow later; what is bounded is its norm over a head.  A
product of a chunk in tf32 parts adds up to 16 steps of three products, each addition losing at most 2^-23 of the
partial sum: 48 2^-23 = 6e-6 of the result's norm at most, its operands' parts 2^-21.  Forward three products follow one another
(K h, T R, K^T U or A U) and T's norm is below 3 for the tests' keys: 3 * 3 * 7e-6 < 1e-4.  The gradients go through
about twice as many: 2e-4.  An element may hold more than its share of the norm: 32 times the root of the mean square.
An output's own rounding adds half a step: 2^-8 (bf16) or 2^-24 (fp32) of the value.

Bounds of the group norm are those of seq_oracle: k 2^-22 times the sum of the terms' absolute values."""
from __future__ import annotations

import math

import numpy as np

from tests import seq_oracle as O

FORWARD, BACKWARD = 1e-4, 2e-4


def check(name, got, ref, bf16, tol, mag=None):
    """Norms and elements of one head's (any slice's) values; mag: the terms' magnitude where they cancel."""
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    if not ref.size:
        return
    assert np.isfinite(got).all(), f"{name}: {int((~np.isfinite(got)).sum())} values are not finite"
    size = np.sqrt(np.mean((np.abs(ref) if mag is None else mag) ** 2)) + 1e-30
    u = 2.0 ** -8 if bf16 else 2.0 ** -24
    off = np.abs(got - ref)
    rms = np.sqrt(np.mean(off ** 2))
    assert rms <= (tol + u) * size, f"{name}: error {rms / size:.3g} of the norm, {tol + u:.3g} allowed"
    worst = (off - u * np.abs(ref)).max()
    assert worst <= 32 * tol * size, f"{name}: an element is {worst / size:.3g} off, {32 * tol:.3g} allowed"


def check_heads(name, got, ref, heads, bf16, tol, mag=None):
    """(T, heads * width): head by head."""
    got, ref = (np.asarray(t).reshape(t.shape[0], heads, t.shape[1] // heads) for t in (got, ref))
    for h in range(heads):
        check(f"{name} head {h}", got[:, h], ref[:, h], bf16, tol, None if mag is None else mag.reshape(got.shape)[:, h])


def delta(q, k, v, g, beta, lens, h0, norm, scale=None, dy=None, dh_out=None):
    """q, k (T, Hk, Dk), v (T, Hv, Dv), g, beta (T, Hv), h0 (S, Hv, Dk, Dv): y, h; with dy the gradients too, and the
    magnitudes of dg's and dbeta's terms."""
    T, Hk, Dk = q.shape
    Hv, Dv = v.shape[1:]
    rep = Hv // Hk
    scale = Dk ** -0.5 if scale is None else scale
    lq, lk = (1 / np.sqrt((t * t).sum(-1, keepdims=True) + 1e-6) if norm else np.ones((T, Hk, 1)) for t in (q, k))
    qn, kn = np.repeat(q * lq, rep, 1), np.repeat(k * lk, rep, 1)
    a = np.exp(g)
    y, left = np.zeros((T, Hv, Dv)), h0.astype(np.float64).copy()
    before, after, rest = (np.zeros((T, Hv, Dk, Dv)) for _ in range(2)), None, np.zeros((T, Hv, Dv))
    hp, hn = before
    for s, (i, j) in enumerate(O.bounds(lens)):
        h = left[s]
        for t in range(i, j):
            hp[t] = np.where(a[t][:, None, None] == 0, 0, a[t][:, None, None] * h)
            rest[t] = v[t] - np.einsum("hkv,hk->hv", hp[t], kn[t])
            h = hp[t] + kn[t][..., None] * (beta[t][:, None] * rest[t])[:, None]
            hn[t] = h
            y[t] = scale * np.einsum("hkv,hk->hv", h, qn[t])
        left[s] = h
    out = {"y": y.reshape(T, Hv * Dv), "h": left}
    if dy is None:
        return out
    dq, dk, dv = np.zeros_like(qn), np.zeros_like(kn), np.zeros_like(v)
    dg, dbeta, mg, mb = (np.zeros((T, Hv)) for _ in range(4))
    dh_in = np.zeros_like(left)
    for s, (i, j) in enumerate(O.bounds(lens)):
        dh = np.zeros_like(left[s]) if dh_out is None else dh_out[s].copy()
        for t in range(j - 1, i - 1, -1):
            u = beta[t][:, None] * rest[t]
            dh = dh + scale * qn[t][..., None] * dy[t][:, None]
            dq[t] = scale * np.einsum("hkv,hv->hk", hn[t], dy[t])
            du = np.einsum("hkv,hk->hv", dh, kn[t])
            dr = beta[t][:, None] * du
            dk[t] = np.einsum("hkv,hv->hk", dh, u) - np.einsum("hkv,hv->hk", hp[t], dr)
            dv[t] = dr
            dbeta[t], mb[t] = (du * rest[t]).sum(-1), np.abs(du * rest[t]).sum(-1)
            dh = dh - kn[t][..., None] * dr[:, None]
            dg[t], mg[t] = (dh * hp[t]).sum((-1, -2)), np.abs(dh * hp[t]).sum((-1, -2))
            dh = a[t][:, None, None] * dh
        dh_in[s] = dh

    def keys(d, x, l):
        d = d.reshape(T, Hk, rep, Dk).sum(2)
        if not norm:
            return d.reshape(T, Hk * Dk), np.abs(d).reshape(T, Hk * Dk)
        # less its part along the vector: for one value all of it, so the error goes with the terms
        m = l * (np.abs(d) + np.abs(x * l) * np.abs(d * x * l).sum(-1, keepdims=True))
        return (l * (d - x * l * (d * x * l).sum(-1, keepdims=True))).reshape(T, Hk * Dk), m.reshape(T, Hk * Dk)

    (gq, mq), (gk, mk) = keys(dq, q, lq), keys(dk, k, lk)
    out.update(dq=gq, dk=gk, mag_dq=mq, mag_dk=mk, dv=dv.reshape(T, Hv * Dv), dg=dg, dbeta=dbeta, dh_in=dh_in,
               mag_dg=mg, mag_dbeta=mb)
    return out


# ----------------------------------------------------------------------------- group norm
def act_of(act, z):
    """The activation, its slope and a bound of its second derivative."""
    if act == "silu":
        return O.silu(z), O.silu_grad(z), 0.5
    if act == "gelu":
        phi = 0.5 * (1 + np.vectorize(math.erf)(z / math.sqrt(2))) if z.size else z
        return z * phi, phi + z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi), 0.8
    return z, np.ones_like(z), 0.0


def gnorm(x, w, b, G, lens, act, eps, dy=None):
    """Outputs and magnitudes: y, stats (S, G, 2); with dy dx, dw, db."""
    T, D = x.shape
    S = len(lens)
    w, b = (np.ones(D) if w is None else w), (np.zeros(D) if b is None else b)
    out, mag = {"y": np.zeros((T, D)), "stats": np.zeros((S, G, 2))}, {"y": np.zeros((T, D))}
    if dy is not None:
        for k, n in (("dx", (T, D)), ("dw", (D,)), ("db", (D,))):
            out[k], mag[k] = np.zeros(n), np.zeros(n)
    for s, (i, j) in enumerate(O.bounds(lens)):
        if j == i:
            continue
        xs = x[i:j].reshape(j - i, G, -1)
        n = xs[:, 0].size
        mean = xs.mean((0, 2), keepdims=True)
        r = 1 / np.sqrt(((xs - mean) ** 2).mean((0, 2), keepdims=True) + eps)
        out["stats"][s] = np.stack([mean[0, :, 0], r[0, :, 0]], -1)
        hat = ((xs - mean) * r).reshape(j - i, D)
        # x less mean: what the roundings of both leave, and of the variance (relative to itself)
        hm = ((np.abs(xs) + np.abs(mean)) * r + np.abs((xs - mean) * r)).reshape(j - i, D)
        z, zm = hat * w + b, hm * np.abs(w) + np.abs(b)
        f, df, second = act_of(act, z)
        out["y"][i:j], mag["y"][i:j] = f, 1.13 * zm
        if dy is None:
            continue
        d, dm = dy[i:j] * df, np.abs(dy[i:j]) * (1.13 + second * zm)
        out["dw"] += (d * hat).sum(0)
        mag["dw"] += (dm * hm).sum(0)
        out["db"] += d.sum(0)
        mag["db"] += dm.sum(0)
        e, em = (d * w).reshape(xs.shape), (dm * np.abs(w)).reshape(xs.shape)
        h3, hm3 = hat.reshape(xs.shape), hm.reshape(xs.shape)
        m1, m2 = e.sum((0, 2), keepdims=True) / n, (e * h3).sum((0, 2), keepdims=True) / n
        out["dx"][i:j] = (r * (e - m1 - h3 * m2)).reshape(j - i, D)
        mag["dx"][i:j] = (r * (em + em.sum((0, 2), keepdims=True) / n + hm3 * (em * hm3).sum((0, 2), keepdims=True) / n)).reshape(j - i, D)
    return out, mag
