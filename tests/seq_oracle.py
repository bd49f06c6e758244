"""The sequence-mixing operators in 64 bits, token by token from their formulas (numpy), with
gradients, and the magnitudes that their error bounds scale with.

Bounds.  Every result is a sum of products; `mag` is the same sum with every term's absolute
value.  A term picks up one rounding (at most 2^-24 relative; 2^-22 for a special-function value,
whose argument's rounding adds |argument| 2^-23) for each operation on its way, so to first order
    |error| <= k 2^-22 mag + u |result|,
where k counts the operations on the longest way: 4 for each token that a state passes, one for
each further term of a sum, and 100 for the functions of one token (softplus, silu and their
derivatives, arguments up to 16); u is the output type's rounding (2^-8 bf16, 2^-24 fp32)."""
from __future__ import annotations

import numpy as np


def sigmoid(v):
    return 0.5 * (1 + np.tanh(0.5 * v))


def silu(v):
    return v * sigmoid(v)


def silu_grad(v):
    s = sigmoid(v)
    return s * (1 + v * (1 - s))


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def bounds(lens):
    out, t = [], 0
    for n in lens:
        out.append((t, t + n))
        t += n
    return out


# --------------------------------------------------------------------------- convolution
def conv(x, w, bias, lens, state, act=True):
    """y, states left, mag of y.  state: (S, W-1, D)."""
    T, D = x.shape
    W = w.shape[1]
    pre, mag = np.zeros((T, D)), np.zeros((T, D))
    left = np.zeros((len(lens), W - 1, D))
    for s, (a, b) in enumerate(bounds(lens)):
        full = np.concatenate([state[s], x[a:b]])
        for t in range(a, b):
            win = full[t - a:t - a + W].T
            pre[t] = bias + (win * w).sum(1)
            mag[t] = np.abs(bias) + np.abs(win * w).sum(1)
        left[s] = full[b - a:]
    if not act:
        return pre, left, mag
    return silu(pre), left, 1.1 * mag


def conv_grad(x, w, bias, lens, state, dy, act=True):
    T, D = x.shape
    W = w.shape[1]
    out = {k: np.zeros(v) for k, v in (("dx", (T, D)), ("dw", (D, W)), ("dbias", (D,)))}
    mag = {k: np.zeros_like(v) for k, v in out.items()}
    for s, (a, b) in enumerate(bounds(lens)):
        full = np.concatenate([state[s], x[a:b]])
        for t in range(a, b):
            win = full[t - a:t - a + W].T
            pre = bias + (win * w).sum(1)
            d = dy[t] * (silu_grad(pre) if act else 1)
            # the slope's own error: its argument's, times a second derivative of at most 1/2
            m = np.abs(dy[t]) * (1.1 + 0.5 * (np.abs(bias) + np.abs(win * w).sum(1)))
            out["dw"] += d[:, None] * win
            mag["dw"] += m[:, None] * np.abs(win)
            out["dbias"] += d
            mag["dbias"] += m
            for j in range(W):
                q = t - W + 1 + j
                if q >= a:
                    out["dx"][q] += w[:, j] * d
                    mag["dx"][q] += np.abs(w[:, j]) * m
    return out, mag


# ---------------------------------------------------------------------------------- scan
def scan(x, dt, A, B, C, G, lens, h0, D=None, z=None, dt_bias=None, act=True, dy=None, dh_out=None):
    """Outputs and their magnitudes: y, h (S, D, N); with dy also the gradients."""
    T, W = x.shape
    N = A.shape[1]
    S = len(lens)
    grp = np.arange(W) // (W // G)
    wide = lambda m: m.reshape(T, G, N)[:, grp]      # noqa: E731   T, W, N
    raw = dt + (0 if dt_bias is None else dt_bias)
    delta = softplus(raw) if act else raw
    dmag = np.abs(delta)
    Bw, Cw = wide(B), wide(C)
    gz = np.ones_like(x) if z is None else silu(z)
    Dv = np.zeros(W) if D is None else D
    a = np.exp(delta[:, :, None] * A)
    u = delta * x
    h, hm = np.zeros((T, W, N)), np.zeros((T, W, N))
    before, beforem = np.zeros((T, W, N)), np.zeros((T, W, N))
    hn, hnm = h0.astype(np.float64).copy(), np.abs(h0)
    for s, (i, j) in enumerate(bounds(lens)):
        v, m = hn[s], hnm[s]
        for t in range(i, j):
            before[t], beforem[t] = v, m
            v = a[t] * v + u[t][:, None] * Bw[t]
            m = a[t] * m + np.abs(u[t][:, None] * Bw[t])
            h[t], hm[t] = v, m
        hn[s], hnm[s] = v, m
    core = (h * Cw).sum(-1) + Dv * x
    corem = (hm * np.abs(Cw)).sum(-1) + np.abs(Dv * x)
    out = {"y": core * gz, "h": hn}
    mag = {"y": corem * np.abs(gz), "h": hnm}
    if dy is None:
        return out, mag
    dyc, dym = dy * gz, np.abs(dy * gz)
    if z is not None:
        out["dz"], mag["dz"] = dy * core * silu_grad(z), np.abs(dy) * corem * (1.1 + 0.5 * np.abs(z))
    g, gm = np.zeros((T, W, N)), np.zeros((T, W, N))
    dh = np.zeros_like(hn) if dh_out is None else dh_out.astype(np.float64).copy()
    dhm = np.abs(dh)
    for s, (i, j) in enumerate(bounds(lens)):
        v, m = dh[s], dhm[s]
        for t in range(j - 1, i - 1, -1):
            g[t] = Cw[t] * dyc[t][:, None] + v
            gm[t] = np.abs(Cw[t]) * dym[t][:, None] + m
            v, m = a[t] * g[t], a[t] * gm[t]
        dh[s], dhm[s] = v, m
    out["dh_in"], mag["dh_in"] = dh, dhm
    q, qm = g * a * before, gm * a * beforem
    gB, gBm = (g * Bw).sum(-1), (gm * np.abs(Bw)).sum(-1)
    dd, ddm = (q * A).sum(-1) + x * gB, (qm * np.abs(A)).sum(-1) + np.abs(x) * gBm
    out["dx"], mag["dx"] = delta * gB + Dv * dyc, dmag * gBm + np.abs(Dv) * dym
    slope = sigmoid(raw) if act else np.ones_like(raw)
    out["ddt"], mag["ddt"] = dd * slope, ddm * slope
    out["ddt_bias"], mag["ddt_bias"] = out["ddt"].sum(0), mag["ddt"].sum(0)
    out["dA"], mag["dA"] = (q * delta[:, :, None]).sum(0), (qm * dmag[:, :, None]).sum(0)
    out["dD"], mag["dD"] = (dyc * x).sum(0), np.abs(dyc * x).sum(0)
    per = lambda m: m.reshape(T, G, W // G, N).sum(2).reshape(T, G * N)   # noqa: E731
    out["dB"], mag["dB"] = per(g * u[:, :, None]), per(gm * np.abs(u)[:, :, None])
    out["dC"], mag["dC"] = per(h * dyc[:, :, None]), per(hm * dym[:, :, None])
    return out, mag


# ---------------------------------------------------------------------------------- norm
def _norm(v, vm, layer, eps):
    """The normalised rows, their magnitude, and 1 / sqrt(...)."""
    if layer:
        mean = v.mean(1, keepdims=True)
        v, vm = v - mean, vm + vm.mean(1, keepdims=True)
    r = 1 / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    # the factor's relative error is that of the values it is computed from
    rel = (np.abs(v) * vm).mean(1, keepdims=True) * r * r
    return v * r, vm * r + np.abs(v * r) * (1 + rel), r


def _norm_back(d, dm, hat, hatm, r, layer):
    c, cm = (d * hat).mean(1, keepdims=True), (dm * hatm).mean(1, keepdims=True)
    m, mm = (d.mean(1, keepdims=True), dm.mean(1, keepdims=True)) if layer else (0, 0)
    grow = 1 + hatm.max(1, keepdims=True) / np.maximum(np.abs(hat).max(1, keepdims=True), 1e-300)
    return r * (d - hat * c - m), r * (dm + hatm * cm + mm) * grow


def norm(x, layer, eps, post, pre, gate=None, after=False, w_post=None, b_post=None, scale=None, res=None, w_pre=None,
         b_pre=None, dy=None, dres_out=None):
    one = lambda v, n=1.0: n if v is None else v      # noqa: E731
    D = x.shape[1]
    out, mag = {}, {}
    gz = silu(gate) if gate is not None else None
    v, vm = x, np.abs(x)
    if gate is not None and not after:
        v, vm = v * gz, vm * np.abs(gz)
    u, um = v, vm
    if post:
        hat, hatm, ru = _norm(v, vm, layer, eps)
        n, nm = hat * one(w_post) + one(b_post, 0), hatm * np.abs(one(w_post)) + np.abs(one(b_post, 0.0))
        u, um = n, nm
    else:
        n, nm = x, np.abs(x)
    if gate is not None and after:
        u, um = u * gz, um * np.abs(gz)
    r, rm = u * one(scale), um * np.abs(one(scale))
    if res is not None:
        r, rm = r + res, rm + np.abs(res)
        out["res_out"], mag["res_out"] = r, rm
    if pre:
        hat2, hat2m, rr = _norm(r, rm, layer, eps)
        out["y"], mag["y"] = hat2 * one(w_pre) + one(b_pre, 0), hat2m * np.abs(one(w_pre)) + np.abs(one(b_pre, 0.0))
    elif res is None:
        out["y"], mag["y"] = r, rm
    if dy is None and dres_out is None:
        return out, mag
    d, dm = np.zeros_like(x), np.zeros_like(x)
    if pre:
        out["dw_pre"], mag["dw_pre"] = (dy * hat2).sum(0), (np.abs(dy) * hat2m).sum(0)
        out["db_pre"], mag["db_pre"] = dy.sum(0), np.abs(dy).sum(0)
        e = dy * one(w_pre)
        d, dm = _norm_back(e, np.abs(e), hat2, hat2m, rr, layer)
    elif res is None:
        d, dm = dy, np.abs(dy)
    if res is not None:
        if dres_out is not None:
            d, dm = d + dres_out, dm + np.abs(dres_out)
        out["dres"], mag["dres"] = d, dm
    out["dscale"], mag["dscale"] = (d * u).sum(0), (dm * um).sum(0)
    d, dm = d * one(scale), dm * np.abs(one(scale))
    if gate is not None and after:
        out["dgate"], mag["dgate"] = d * n * silu_grad(gate), dm * nm * (1.1 + 0.5 * np.abs(gate))
        d, dm = d * gz, dm * np.abs(gz)
    if post:
        out["dw_post"], mag["dw_post"] = (d * hat).sum(0), (dm * hatm).sum(0)
        out["db_post"], mag["db_post"] = d.sum(0), dm.sum(0)
        d, dm = _norm_back(d * one(w_post), dm * np.abs(one(w_post)), hat, hatm, ru, layer)
    if gate is not None and not after:
        out["dgate"], mag["dgate"] = d * x * silu_grad(gate), dm * np.abs(x) * (1.1 + 0.5 * np.abs(gate))
        d, dm = d * gz, dm * np.abs(gz)
    out["dx"], mag["dx"] = d, dm
    return out, mag


def check(name, got, ref, mag, k, bf16):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    u = 2.0 ** -8 if bf16 else 2.0 ** -24
    tol = k * 2.0 ** -22 * mag + u * np.abs(ref) + 1e-36
    bad = ~(np.abs(got - ref) <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - ref) / tol, 0)), ref.shape)
        raise AssertionError(f"{name}: {int(bad.sum())}/{ref.size} outside the bound; worst at {i}: got {got[i]!r}, "
                             f"64 bits {ref[i]!r}, tolerance {tol[i]!r}")


# ------------------------------------------------------------------- cases of long memory
def slow_case(rng, lens, D, N):
    """Inputs of a scan whose states remember thousands of tokens: steps of 1e-3 to 1e-2 and A of -1 to -0.05.  x is zero
    but at a sequence's beginning and a few tokens, dy but at its end and a few: what reaches the others comes a
    long way.  For softplus without a bias."""
    T, S = sum(lens), len(lens)
    x, dy = rng.standard_normal((T, D)), rng.standard_normal((T, D))
    keep = np.zeros(T, bool), np.zeros(T, bool)
    for a, b in bounds(lens):
        keep[0][a:min(a + 40, b)] = True
        keep[1][max(b - 40, a):b] = True
        keep[0][a + 499:b:997] = True
        keep[1][a + 250:b:997] = True
    x[~keep[0]] = 0
    dy[~keep[1]] = 0
    step = np.exp(rng.uniform(np.log(1e-3), np.log(1e-2), (T, D)))
    return dict(x=x, dt=np.log(np.expm1(step)), A=-rng.uniform(0.05, 1, (D, N)), B=rng.standard_normal((T, N)), C=rng.standard_normal((T, N)),
                D=rng.standard_normal(D)), dict(h=rng.standard_normal((S, D, N)), dy=dy, dh=rng.standard_normal((S, D, N)))


def scan_in_pieces(x, dt, A, B, C, D, lens, h0, piece, parts, fault=None):
    """y and the states left (one group, softplus, no gate) as the library forms them: every piece of `piece` tokens
    from a zero state, the pieces' results joined in `parts` parts, every piece again from the state before it.
    `fault` plants a mistake in the joining."""
    T, W = x.shape
    delta = softplus(dt)
    a, add = np.exp(delta[:, :, None] * A), (delta * x)[:, :, None] * B[:, None]
    begin = {i: s for s, (i, j) in enumerate(bounds(lens)) if j > i}
    end = {j - 1: s for s, (i, j) in enumerate(bounds(lens)) if j > i}
    count = (T + piece - 1) // piece
    e, total, cut = [], [], []
    for r in range(count):
        h, t_sum, stop = np.zeros((W, A.shape[1])), np.zeros(W), False
        for t in range(r * piece, min(T, (r + 1) * piece)):
            if t in begin:
                h, t_sum, stop = h0[begin[t]], np.zeros(W), True
            h, t_sum = a[t] * h + add[t], t_sum + delta[t]
        e.append(h), total.append(t_sum), cut.append(stop)

    def step(c, e, total, stop):
        return e if stop and fault != "ends of sequences" else e + np.exp(total[:, None] * A) * c

    length = -(-count // parts)
    before, result = [], []
    for q in range(parts):
        rs = range(q * length, min(count, (q + 1) * length))
        c, t_sum, stop = np.zeros_like(e[0]), np.zeros(W), False
        for r in rs:
            c, t_sum, stop = step(c, e[r], total[r], cut[r]), np.zeros(W) if cut[r] else t_sum + total[r], stop or cut[r]
        result.append((c, t_sum, stop))
        c = np.zeros_like(e[0])
        for k in range(q):
            if fault == "parts before" or (fault == "older parts" and k < q - 1):
                continue
            c = step(c, result[k][0], result[k][1] * (fault != "decay over a part"), result[k][2])
        for r in rs:
            before.append(c)
            c = step(c, e[r], total[r], cut[r])
    y, left = np.zeros_like(x), h0.copy()
    for r in range(count):
        h = before[r]
        for t in range(r * piece, min(T, (r + 1) * piece)):
            if t in begin:
                h = h0[begin[t]]
            h = a[t] * h + add[t]
            y[t] = (h * C[t]).sum(-1) + D * x[t]
            if t in end:
                left[end[t]] = h
    return y, left
