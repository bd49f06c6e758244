"""The gated delta rule and the group norm with an activation, on sizes that stand for their use.
Each has a plain form (elementary torch operations in 32 bits) and the library's call; `own`
selects between them.

  delta  per value head: h' = exp(g_t) h_{t-1}; u = beta_t (v_t - h'^T k_t); h_t = h' + k_t u^T;
         y_t = h_t^T q_t / sqrt(Dk).  Value heads share the key heads' q and k.  With "norm", q and k
         are divided by their lengths first.  h_0 comes from the sequence's state (or is zero)
  gnorm  z = (x - mean) rstd w + b over the tokens of a sequence (the pixels of an image) and the
         channels of a group; y = act(z)

A case's "way" is step (one token per sequence), prompt (forward; the delta rule's states in and
out) or train (forward and backward).  Ragged cases pack sequences of unequal lengths.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS_QK = 1e-6
EPS_GN = 1e-5
CHUNK = 64


# --------------------------------------------------------------------------------- the cases
def listed():
    def delta(name, way, dtype, S, T, Hk, Hv, Dk, Dv, norm=True, ragged=False):
        return dict(name=name, op="delta", way=way, dtype=dtype, S=S, T=T, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv, norm=norm,
                    ragged=ragged)

    def gnorm(name, way, dtype, S, T, D, G, act, ragged=False):
        return dict(name=name, op="gnorm", way=way, dtype=dtype, S=S, T=T, D=D, G=G, act=act, ragged=ragged)

    return [
        # one decoding step of four users: latency alone
        delta("delta_step_bf16_n4_h16", "step", "bf16", 4, 4, 16, 16, 128, 128),
        # one decoding step of a full serving batch, keys shared by two value heads: bound by the states' bytes
        delta("delta_step_bf16_n256_h32", "step", "bf16", 256, 256, 16, 32, 128, 128),
        # one user's prompt: few heads, a long axis
        delta("delta_prompt_bf16_l2048_h16", "prompt", "bf16", 1, 2048, 16, 16, 128, 128),
        # a serving batch of prompts of unequal lengths, packed, with their cached states
        delta("delta_prompt_bf16_ragged_h32", "prompt", "bf16", 13, 6011, 16, 32, 128, 128, ragged=True),
        # packed prompts in 32 bits, odd head sizes, keys that come with unit length
        delta("delta_prompt_f32_ragged_k48_v80", "prompt", "f32", 7, 5003, 3, 6, 48, 80, norm=False, ragged=True),
        # a small model's training step in 32 bits
        delta("delta_train_f32_n2_l1500_h6", "train", "f32", 2, 3000, 6, 6, 64, 64),
        # a large training batch
        delta("delta_train_bf16_n4_l2048_h32", "train", "bf16", 4, 4 * 2048, 16, 32, 128, 128),
        # one sample of 1500 audio frames: latency
        gnorm("gnorm_prompt_bf16_n1_l1500_d384", "prompt", "bf16", 1, 1500, 384, 32, "silu"),
        # images between two convolutions of 512 channels
        gnorm("gnorm_prompt_bf16_n16_56x56_d512", "prompt", "bf16", 16, 16 * 56 * 56, 512, 32, "silu"),
        # packed clips of unequal lengths in 32 bits, 55 channels a group
        gnorm("gnorm_prompt_f32_ragged_d770_g14", "prompt", "f32", 7, 5003, 770, 14, "gelu", ragged=True),
        # an audio model's training step: every channel a group of its own
        gnorm("gnorm_train_f32_n8_l1500_d1280", "train", "f32", 8, 8 * 1500, 1280, 1280, "gelu"),
        # a large training batch of images
        gnorm("gnorm_train_bf16_n32_56x56_d512", "train", "bf16", 32, 32 * 56 * 56, 512, 32, "silu"),
    ]


def _odd(rng, lo, hi, step=1):
    """A size from lo to hi, uniform in its logarithm: an odd multiple of `step`."""
    v = int(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi)))))
    return max(1, v // step | 1) * step


def draw(rng):
    dtype = rng.choice(["bf16", "f32"])
    if rng.random() < 0.4:
        way = rng.choice(["prompt", "train"])
        G = rng.choice([1, 4, 8, 16, 32, 32, 0])               # 0: every channel a group of its own
        D = max(1, _odd(rng, 32, 2048) // max(G, 1)) * max(G, 1) if rng.random() < 0.4 else rng.choice(
            [128, 256, 384, 512, 768, 1024, 1280])
        c = dict(op="gnorm", way=way, dtype=dtype, D=D, G=G or D, act=rng.choice(["none", "silu", "silu", "gelu"]),
                 ragged=rng.random() < 0.4)
        most = (1 << 24) // D
        if c["ragged"]:
            c["S"] = _odd(rng, 1, 24)
            c["T"] = max(c["S"], _odd(rng, 16, min(20000, most // 4)))
        else:
            c["S"] = _odd(rng, 1, 32)
            c["T"] = c["S"] * _odd(rng, 1, max(1, min(16384, most // c["S"])))
        return c
    way = rng.choice(["step", "prompt", "prompt", "train"])
    Hk = _odd(rng, 1, 16)
    c = dict(op="delta", way=way, dtype=dtype, Hk=Hk, Hv=Hk * rng.choice([1, 1, 2, 3]),
             Dk=rng.choice([32, 64, 64, 96, 128, 128, _odd(rng, 8, 128), 2 * _odd(rng, 4, 64)]),
             Dv=rng.choice([32, 64, 64, 96, 128, 128, 256, _odd(rng, 8, 200), 8 * _odd(rng, 1, 24)]),
             norm=rng.random() < 0.7)
    size = c["Hv"] * max(64, c["Dk"]) * max(64, c["Dv"])
    if way == "step":
        c["S"] = c["T"] = _odd(rng, 1, min(400, (1 << 26) // size))
        c["ragged"] = False
        return c
    most = max(64, (1 << (30 if way == "train" else 31)) // size)
    c["ragged"] = rng.random() < 0.5
    if c["ragged"]:
        c["S"] = _odd(rng, 1, 16)
        c["T"] = max(c["S"], _odd(rng, 16, min(8192, max(64, most // 4))))
    else:
        c["S"] = _odd(rng, 1, 8)
        c["T"] = c["S"] * _odd(rng, 1, max(1, min(8192, most // c["S"])))
    return c


def lengths(case):
    """Sequence lengths of a case: equal ones, or (ragged) unequal ones that hold an empty
    sequence and a single token wherever there is room."""
    S, T = case["S"], case["T"]
    if not case["ragged"]:
        return [T // S] * S
    r = random.Random(1000003 * S + T)
    share = [r.random() ** 2 + 1e-3 for _ in range(S)]
    lens = [int(T * v / sum(share)) for v in share]
    if S > 2:
        lens[S // 2], lens[S // 3] = 0, 1
    lens[lens.index(max(lens))] += T - sum(lens)
    return lens


# ------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    S, T, way = case["S"], case["T"], case["way"]
    dt = DT[case["dtype"]]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=gen, device=dev) * (hi - lo) + lo

    s = dict(case=case, lens=lengths(case), starts=None)
    if case["ragged"]:
        s["starts"] = torch.tensor([0] + torch.tensor(s["lens"]).cumsum(0).tolist(), dtype=torch.int32, device=dev)
    if case["op"] == "gnorm":
        D = case["D"]
        # what a convolution with a bias leaves: channels of unequal means and spreads
        s["x"] = (torch.randn(T, D, generator=gen, device=dev) * uniform(D, lo=0.5, hi=2.0) + normal(D, dtype=torch.float32)).to(dt)
        s["w"] = uniform(D, lo=0.5, hi=1.5).to(dt)
        s["b"] = normal(D, std=0.2)
        if way == "train":
            s["dy"] = normal(T, D)
        if own:
            _own_gnorm(s)
        return s

    Hk, Hv, Dk, Dv = case["Hk"], case["Hv"], case["Dk"], case["Dv"]
    # one tensor holds q, k and v side by side, as the short convolution's silu leaves them
    a = torch.randn(T, 2 * Hk * Dk + Hv * Dv, generator=gen, device=dev)
    a = a / (1 + torch.exp(-a))
    if not case["norm"]:
        qk = a[:, :2 * Hk * Dk].view(T, 2 * Hk, Dk)
        qk /= torch.sqrt((qk * qk).sum(-1, keepdim=True) + EPS_QK)
    a = a.to(dt)
    s["q"], s["k"], s["v"] = a[:, :Hk * Dk], a[:, Hk * Dk:2 * Hk * Dk], a[:, 2 * Hk * Dk:]
    # decay factors: a rate for each head, a step for each token
    step = torch.exp(uniform(Hv, lo=math.log(1e-3), hi=math.log(1e-1)))
    raw = normal(T, Hv, dtype=torch.float32) + step + torch.log(-torch.expm1(-step))
    s["g"] = -uniform(Hv, lo=1.0, hi=16.0) * torch.log1p(torch.exp(raw))
    s["beta"] = 1 / (1 + torch.exp(-normal(T, Hv, dtype=torch.float32)))
    s["h"] = normal(S, Hv, Dk, Dv, std=0.2, dtype=torch.float32) if way != "train" else None
    if way == "train":
        s["dy"] = normal(T, Hv * Dv)
    if own:
        _own_delta(s)
    return s


# ----------------------------------------------------------------------- the library's own calls
def _code(case):
    from convolution_forward_implicit_gb300.binding import CONV_BF16, CONV_F32
    return {"bf16": CONV_BF16, "f32": CONV_F32}[case["dtype"]]


def _own_delta(s):
    from convolution_forward_implicit_gb300 import delta
    c = s["case"]
    S, T, Hk, Hv, Dk, Dv = (c[k] for k in ("S", "T", "Hk", "Hv", "Dk", "Dv"))
    new = lambda *shape, dtype=s["q"].dtype: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    kw = dict(ragged=c["ragged"], qk_norm=c["norm"])
    s["plan"] = delta.SeqDeltaPlan(S, T, Hk, Hv, Dk, Dv, _code(c), "step" if c["way"] == "step" else "fwd", **kw).allocate()
    s["y"] = new(T, Hv * Dv)
    if c["way"] == "train":
        s["bwd"] = delta.SeqDeltaPlan(S, T, Hk, Hv, Dk, Dv, _code(c), "bwd", **kw).allocate()
        s["saved"] = s["bwd"].allocate_saved()
        s["dq"], s["dk"], s["dv"] = new(T, Hk * Dk), new(T, Hk * Dk), new(T, Hv * Dv)
        s["dg"], s["dbeta"] = new(T, Hv, dtype=torch.float32), new(T, Hv, dtype=torch.float32)
    else:
        s["h_out"] = new(S, Hv, Dk, Dv, dtype=torch.float32)


def _own_gnorm(s):
    from convolution_forward_implicit_gb300 import gnorm
    c = s["case"]
    S, T, D, G = c["S"], c["T"], c["D"], c["G"]
    kw = dict(ragged=c["ragged"], act=c["act"], eps=EPS_GN)
    s["plan"] = gnorm.SeqGroupNormPlan(S, T, D, G, _code(c), "fwd", **kw).allocate()
    s["y"], s["stats"] = torch.empty_like(s["x"]), None
    if c["way"] == "train":
        s["bwd"] = gnorm.SeqGroupNormPlan(S, T, D, G, _code(c), "bwd", **kw).allocate()
        s["stats"] = torch.empty(S, G, 2, device="cuda")
        s["dx"] = torch.empty_like(s["x"])
        s["dw"], s["db"] = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")


def _run_own(s):
    c = s["case"]
    if c["op"] == "gnorm":
        s["plan"].forward(s["x"], s["y"], w=s["w"], b=s["b"], starts=s["starts"], stats=s["stats"])
        out = {"y": s["y"]}
        if c["way"] == "train":
            s["bwd"].backward(s["x"], s["stats"], s["dy"], s["dx"], w=s["w"], b=s["b"], dw=s["dw"], db=s["db"],
                              starts=s["starts"])
            out.update(dx=s["dx"], dw=s["dw"], db=s["db"])
        return out
    a = (s["q"], s["k"], s["v"], s["g"], s["beta"])
    if c["way"] == "step":
        s["plan"].step(*a, s["h"], s["h_out"], s["y"])
        return {"y": s["y"], "h": s["h_out"]}
    if c["way"] == "prompt":
        s["plan"].forward(*a, s["y"], starts=s["starts"], h_in=s["h"], h_out=s["h_out"])
        return {"y": s["y"], "h": s["h_out"]}
    s["plan"].forward(*a, s["y"], starts=s["starts"], saved=s["saved"])
    s["bwd"].backward(*a, s["dy"], s["saved"], s["dq"], s["dk"], s["dv"], s["dg"], s["dbeta"], starts=s["starts"])
    return {k: s[k] for k in ("y", "dq", "dk", "dv", "dg", "dbeta")}


# ----------------------------------------------------------------------------- the plain forms
def _padded(lens, T, to, dev):
    """Token indices of every sequence, padded with T to a multiple of `to`, and where tokens are."""
    n = torch.tensor(lens, device=dev)
    most = max(1, -(-max(lens) // to)) * to
    pos = torch.arange(most, device=dev)
    there = pos < n[:, None]
    return torch.where(there, (n.cumsum(0) - n)[:, None] + pos, T), there


def _inverse(L):
    """(I + L)^-1 of strictly lower triangular matrices: [[P, 0], [B, Q]]^-1 = [[P', 0], [-Q' B P', Q']],
    for blocks of 1, 2, 4, ... rows."""
    n = L.shape[-1]
    i = torch.arange(n, device=L.device)
    inv, size = torch.eye(n, device=L.device).expand_as(L), 1
    while size < n:
        left = (i[:, None] // size % 2 == 1) & (i[:, None] // size == i // size + 1)
        inv = inv - inv @ (L * left) @ inv
        size *= 2
    return inv


def _delta(c, idx, there, q, k, v, g, beta, h):
    """y of every token and the states left; the tokens of a chunk at once, chunk after chunk."""
    S, T, Hk, Hv, Dk, Dv = (c[n] for n in ("S", "T", "Hk", "Hv", "Dk", "Dv"))
    if c["norm"]:
        q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + EPS_QK)
        k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + EPS_QK)

    def chunks(t):                                  # T, heads, ... -> S, heads, chunks, CHUNK, ...
        t = torch.cat([t, t.new_zeros(1, *t.shape[1:])])[idx]
        return t.view(S, -1, CHUNK, *t.shape[2:]).movedim(3, 1)

    q, k = (chunks(t.repeat_interleave(Hv // Hk, 1)) for t in (q / math.sqrt(Dk), k))
    v, g, beta = chunks(v), chunks(g), chunks(beta)[..., None]
    b = g.cumsum(-1)
    i = torch.arange(CHUNK, device=b.device)
    E = torch.exp(torch.where(i[:, None] >= i, b[..., :, None] - b[..., None, :], -math.inf))
    kt = k.transpose(-1, -2)
    inv = _inverse(beta * E * (k @ kt) * (i[:, None] > i))
    U0, W = inv @ (beta * v), inv @ (beta * torch.exp(b)[..., None] * k)
    A, qb = E * (q @ kt), torch.exp(b)[..., None] * q
    end = b[..., -1:]
    ket, last = (torch.exp(end - b)[..., None] * k).transpose(-1, -2), torch.exp(end)[..., None]
    y = []
    for n in range(b.shape[2]):                     # every chunk starts from the state the one before it left
        U = U0[:, :, n] - W[:, :, n] @ h
        y.append(qb[:, :, n] @ h + A[:, :, n] @ U)
        h = last[:, :, n] * h + ket[:, :, n] @ U
    y = torch.stack(y, 2).movedim(1, 3).reshape(S, -1, Hv, Dv)
    return y[there], h


def _plain_delta(s):
    c, dt = s["case"], s["q"].dtype
    S, T, Hk, Hv, Dk, Dv = (c[n] for n in ("S", "T", "Hk", "Hv", "Dk", "Dv"))
    q, k, v = s["q"].reshape(T, Hk, Dk).float(), s["k"].reshape(T, Hk, Dk).float(), s["v"].reshape(T, Hv, Dv).float()
    g, beta = s["g"], s["beta"]
    if c["way"] == "step":
        if c["norm"]:
            q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + EPS_QK)
            k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + EPS_QK)
        q, k = (t.repeat_interleave(Hv // Hk, 1)[..., None] for t in (q / math.sqrt(Dk), k))
        h = torch.exp(g)[..., None, None] * s["h"]
        u = beta[..., None] * (v - (h * k).sum(2))
        h = h + k * u[:, :, None]
        return {"y": (h * q).sum(2).to(dt).view(T, -1), "h": h}
    idx, there = _padded(s["lens"], T, CHUNK, q.device)
    if c["way"] == "prompt":
        y, h = _delta(c, idx, there, q, k, v, g, beta, s["h"])
        return {"y": y.to(dt).reshape(T, -1), "h": h}
    ins = [t.detach().requires_grad_() for t in (q, k, v, g, beta)]
    y, _ = _delta(c, idx, there, *ins, q.new_zeros(S, Hv, Dk, Dv))
    d = torch.autograd.grad(y, ins, s["dy"].float().view(T, Hv, Dv))
    out = {"y": y.detach().to(dt).reshape(T, -1)}
    out.update({n: t.to(dt).reshape(T, -1) for n, t in zip(("dq", "dk", "dv"), d)})
    out.update(dg=d[3], dbeta=d[4])
    return out


def _act(c, z):
    """The activation of z and its slope."""
    if c["act"] == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return z * sig, sig * (1 + z * (1 - sig))
    if c["act"] == "gelu":
        phi = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * phi, phi + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return z, torch.ones_like(z)


def _plain_gnorm(s):
    c, dt = s["case"], s["x"].dtype
    S, T, D, G = c["S"], c["T"], c["D"], c["G"]
    x, w, b = s["x"].float(), s["w"].float(), s["b"].float()
    if c["ragged"]:
        idx, there = _padded(s["lens"], T, 1, x.device)
        rows = lambda t: torch.cat([t, t.new_zeros(1, D)])[idx].view(S, -1, G, D // G)       # noqa: E731
        back = lambda t: t.reshape(S, -1, D)[there]                                             # noqa: E731
        mask = there[:, :, None, None]
        n = torch.tensor(s["lens"], device=x.device).clamp(min=1).view(S, 1, 1, 1) * (D // G)
    else:
        rows = lambda t: t.view(S, -1, G, D // G)                                               # noqa: E731
        back = lambda t: t.reshape(T, D)                                                        # noqa: E731
        mask, n = 1.0, T // S * (D // G)
    x = rows(x)
    mean = x.sum((1, 3), keepdim=True) / n
    x = (x - mean) * mask
    rstd = 1 / torch.sqrt((x * x).sum((1, 3), keepdim=True) / n + EPS_GN)
    x = x * rstd
    w = w.view(G, D // G)
    y, slope = _act(c, x * w + b.view(G, D // G))
    out = {"y": back(y).to(dt)}
    if c["way"] == "train":
        dz = rows(s["dy"].float()) * slope
        out["dw"], out["db"] = (dz * x).sum((0, 1)).view(D), dz.sum((0, 1)).view(D)
        dn = dz * w
        dx = rstd * (dn - dn.sum((1, 3), keepdim=True) / n - x * ((dn * x).sum((1, 3), keepdim=True) / n))
        out["dx"] = back(dx).to(dt)
    return out


def run(state):
    if own:
        return _run_own(state)
    return _plain_delta(state) if state["case"]["op"] == "delta" else _plain_gnorm(state)


# --------------------------------------------------------------------- the definition in 64 bits
def _exact_delta(s):
    """Token by token, all sequences side by side; backward from states kept at every 64th token."""
    c = s["case"]
    S, T, Hk, Hv, Dk, Dv = (c[n] for n in ("S", "T", "Hk", "Hv", "Dk", "Dv"))
    dev, f64 = s["q"].device, torch.float64
    rep = Hv // Hk
    q0, k0 = (s[n].to(f64).reshape(T, Hk, Dk) for n in ("q", "k"))
    lq, lk = ((t.square().sum(-1, keepdim=True) + EPS_QK).rsqrt() if c["norm"] else torch.ones(T, Hk, 1, dtype=f64, device=dev)
              for t in (q0, k0))
    one = lambda t: torch.cat([t, torch.zeros_like(t[:1])])                 # noqa: E731   row T: no token
    q, k = (one((t * l).repeat_interleave(rep, 1)) for t, l in ((q0, lq), (k0, lk)))
    v, g, beta = one(s["v"].to(f64).reshape(T, Hv, Dv)), one(s["g"].to(f64)), one(s["beta"].to(f64))
    n = torch.tensor(s["lens"], device=dev)
    first = n.cumsum(0) - n
    token = lambda p: torch.where(p < n, first + p, torch.full_like(n, T))  # noqa: E731
    scale = Dk ** -0.5
    h = s["h"].to(f64) if s["h"] is not None else torch.zeros(S, Hv, Dk, Dv, dtype=f64, device=dev)
    most = max(s["lens"])
    y = torch.zeros(T + 1, Hv, Dv, dtype=f64, device=dev)

    def forward(h, p):
        t = token(p)
        hp = h * g[t].exp()[..., None, None]
        r = v[t] - torch.einsum("shkv,shk->shv", hp, k[t])
        return t, hp, r, hp + k[t][..., None] * (beta[t][..., None] * r)[:, :, None]

    kept = []
    for p in range(most):
        if p % 64 == 0 and c["way"] == "train":
            kept.append(h)
        t, _, _, h = forward(h, p)
        y[t] = torch.einsum("shkv,shk->shv", h, q[t]) * scale
    out = {"y": y[:T].reshape(T, -1)}
    if c["way"] != "train":
        out["h"] = h
        return out
    dy = one(s["dy"].to(f64).reshape(T, Hv, Dv))
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, dbeta = torch.zeros_like(g), torch.zeros_like(beta)
    dh = torch.zeros_like(h)
    for start in range((most - 1) // 64 * 64, -1, -64):
        h, part = kept[start // 64], []
        for p in range(start, min(start + 64, most)):
            t, hp, r, h = forward(h, p)
            part.append((t, hp, r, h))
        for t, hp, r, h in reversed(part):
            u = beta[t][..., None] * r
            dh = dh + scale * q[t][..., None] * dy[t][:, :, None]
            dq[t] = scale * torch.einsum("shkv,shv->shk", h, dy[t])
            du = torch.einsum("shkv,shk->shv", dh, k[t])
            dr = beta[t][..., None] * du
            dk[t] = torch.einsum("shkv,shv->shk", dh, u) - torch.einsum("shkv,shv->shk", hp, dr)
            dv[t], dbeta[t] = dr, (du * r).sum(-1)
            dh = dh - k[t][..., None] * dr[:, :, None]
            dg[t] = (dh * hp).sum((-1, -2))
            dh = dh * g[t].exp()[..., None, None]

    def keys(d, x, l):                      # the sum over the value heads that share a key head; the length's part
        d = d[:T].view(T, Hk, rep, Dk).sum(2)
        return (l * (d - x * l * (d * x * l).sum(-1, keepdim=True)) if c["norm"] else d).reshape(T, -1)

    out.update(dq=keys(dq, q0, lq), dk=keys(dk, k0, lk), dv=dv[:T].reshape(T, -1), dg=dg[:T], dbeta=dbeta[:T])
    return out


def _exact_gnorm(s):
    """Sequence by sequence; the gradients from the formulas of the mean and the variance."""
    c = s["case"]
    T, D, G = c["T"], c["D"], c["G"]
    x, w, b = (s[n].double() for n in ("x", "w", "b"))
    y = torch.zeros_like(x)
    train = c["way"] == "train"
    if train:
        dy, dx, dw, db = s["dy"].double(), torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(b)
    at = 0
    for n in s["lens"]:
        if n:
            xs = x[at:at + n].reshape(n, G, D // G)
            var, mean = torch.var_mean(xs, dim=(0, 2), unbiased=False, keepdim=True)
            r = (var + EPS_GN).rsqrt()
            xh = ((xs - mean) * r).reshape(n, D)
            z = xh * w + b
            if c["act"] == "silu":
                sg = torch.sigmoid(z)
                f, df = z * sg, sg + z * sg * (1 - sg)
            elif c["act"] == "gelu":
                cdf = torch.special.ndtr(z)
                f, df = z * cdf, cdf + z * torch.exp(-z * z / 2) * (2 * math.pi) ** -0.5
            else:
                f, df = z, torch.ones_like(z)
            y[at:at + n] = f
            if train:
                dz = dy[at:at + n] * df
                dw += (dz * xh).sum(0)
                db += dz.sum(0)
                dxs, xg = (dz * w).reshape(n, G, D // G), xh.reshape(n, G, D // G)
                dvar = (dxs * xg).mean((0, 2), keepdim=True)
                dx[at:at + n] = (r * (dxs - dxs.mean((0, 2), keepdim=True) - xg * dvar)).reshape(n, D)
        at += n
    return {"y": y, "dx": dx, "dw": dw, "db": db} if train else {"y": y}


def exact(case, seed):
    if case["op"] == "delta" and max(lengths(case)) > 16384:
        return None
    s = prepare(case, seed)
    return _exact_delta(s) if case["op"] == "delta" else _exact_gnorm(s)


def work(case):
    """Each input read once and each output written once; the operations of the recurrence itself."""
    S, T, e = case["S"], case["T"], 2 if case["dtype"] == "bf16" else 4
    train = case["way"] == "train"
    if case["op"] == "gnorm":
        n = T * case["D"]
        return {"bytes": n * e * (4 if train else 2) + case["D"] * (2 * e + 8 * train), "flops": n * (30 if train else 12)}
    Hk, Hv, Dk, Dv = (case[n] for n in ("Hk", "Hv", "Dk", "Dv"))
    ins, y = T * e * (2 * Hk * Dk + Hv * Dv) + T * Hv * 8, T * e * Hv * Dv
    core = T * Hv * Dk * Dv
    if train:
        return {"bytes": 2 * ins + 2 * y, "flops": 20 * core}
    return {"bytes": ins + y + 8 * S * Hv * Dk * Dv, "flops": 6 * core}
