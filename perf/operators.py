"""The sequence-mixing operators on sizes that stand for their use: the short causal depthwise
convolution, the selective state space scan it feeds, and the norm, gate, residual step around
such a block.  Each has a plain form (elementary torch operations in 32 bits) and the
library's call; `own` selects between them.

  conv   y[t,d] = silu(bias[d] + sum_j w[d,j] x[t-W+1+j, d]) within a sequence; the W-1 inputs
         before a sequence's first token come from its state (or are zero)
  scan   delta = softplus(dt + dt_bias); h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t;
         y_t = (C_t . h_t + D x_t) silu(z_t); h_0 comes from the sequence's state (or is zero)
  norm   u = [norm(x silu(gate)) w_post + b_post]; r = res + scale u; y = norm(r) w_pre + b_pre

A case's "way" is step (one token per sequence), prompt (forward, states in and out) or train
(forward and backward).  Ragged cases pack sequences of unequal lengths, empty ones among them.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------------- the cases
def listed():
    def conv(name, way, dtype, S, T, D, W=4, ragged=False):
        return dict(name=name, op="conv", way=way, dtype=dtype, S=S, T=T, D=D, W=W, ragged=ragged)

    def scan(name, way, dtype, S, T, D, N=16, G=1, ragged=False):
        return dict(name=name, op="scan", way=way, dtype=dtype, S=S, T=T, D=D, N=N, G=G, ragged=ragged)

    def norm(name, way, dtype, res, T, D, kind, post, gate, pre, scale):
        return dict(name=name, op="norm", way=way, dtype=dtype, res=res, T=T, D=D, kind=kind, post=post, gate=gate,
                    pre=pre, scale=scale)

    return [
        # one decoding step of four users: latency alone
        conv("conv_step_bf16_n4_d1536", "step", "bf16", 4, 4, 1536),
        # a serving batch of prompts of unequal lengths, packed, with their cached states
        conv("conv_prompt_bf16_ragged_d2560", "prompt", "bf16", 13, 6011, 2560, ragged=True),
        # an audio model's training step: 1500 frames, 1280 channels, 32 bits
        conv("conv_train_f32_n8_l1500_d1280", "train", "f32", 8, 8 * 1500, 1280),
        # a large training batch
        conv("conv_train_bf16_n8_l2048_d4096", "train", "bf16", 8, 8 * 2048, 4096),
        # one decoding step of four users
        scan("scan_step_bf16_n4_d1536", "step", "bf16", 4, 4, 1536),
        # one decoding step of a full serving batch: bound by the states' bytes
        scan("scan_step_bf16_n256_d4096", "step", "bf16", 256, 256, 4096),
        # one user's prompt: few channels, a long axis
        scan("scan_prompt_bf16_l2048_d2048", "prompt", "bf16", 1, 2048, 2048),
        # packed prompts in 32 bits, odd channel and state counts, two groups of B and C
        scan("scan_prompt_f32_ragged_d770_n12", "prompt", "f32", 7, 5003, 770, N=12, G=2, ragged=True),
        # a training batch
        scan("scan_train_bf16_n4_l2048_d4096", "train", "bf16", 4, 4 * 2048, 4096),
        # the norm between two blocks while decoding for four users, 32-bit residual stream
        norm("norm_step_bf16_n4_d2048", "step", "bf16", "f32", 4, 2048, "rms", False, False, True, False),
        # a training batch with everything on: gated norm after the block, scaled residual, next norm
        norm("norm_train_bf16_t8192_d4096", "train", "bf16", "f32", 8192, 4096, "rms", True, True, True, True),
        # a convolution block's layer norm and layer scale in 32 bits, odd row count
        norm("norm_train_f32_t6007_d1280", "train", "f32", "f32", 6007, 1280, "layer", False, False, True, True),
    ]


def _odd(rng, lo, hi, step=1):
    """A size from lo to hi, uniform in its logarithm: an odd multiple of `step`."""
    v = int(math.exp(rng.uniform(math.log(lo), math.log(hi))))
    return max(1, v // step | 1) * step


def _width(rng):
    return rng.choice([rng.choice([384, 512, 768, 1024, 1280, 1536, 2048, 2560, 4096]), _odd(rng, 64, 4096, 8),
                       _odd(rng, 64, 4096)])


def draw(rng):
    op = rng.choice(["conv", "scan", "norm"])
    way = rng.choice(["step", "prompt", "train"]) if op != "norm" else rng.choice(["step", "train"])
    dtype = rng.choice(["bf16", "f32"])
    D = _width(rng)
    if op == "norm":
        T = _odd(rng, 1, 300) if way == "step" else _odd(rng, 300, min(32768, (1 << 25) // D))
        post, pre = rng.choice([(False, True), (True, False), (True, True)])
        return dict(op=op, way=way, dtype=dtype, res=rng.choice([dtype, "f32"]), T=T, D=D,
                    kind=rng.choice(["rms", "layer"]), post=post, gate=post and rng.random() < 0.5, pre=pre,
                    scale=rng.random() < 0.5)
    c = dict(op=op, way=way, dtype=dtype, D=D)
    per = 1
    if op == "conv":
        c["W"] = rng.choice([2, 3, 4, 4, 5])
    else:
        c["N"] = rng.choice([4, 8, 16, 16, 16, 24, 32, 64])
        c["G"] = rng.choice([1, 1, 2]) if D % 2 == 0 else 1
        per = c["N"]
    if way == "step":
        c["S"] = c["T"] = _odd(rng, 1, 400 if per <= 16 else 100)
        c["ragged"] = False
        return c
    most = (1 << 26) // D if op == "conv" else (1 << 29) // (D * per)
    c["ragged"] = rng.random() < 0.5
    if c["ragged"]:
        c["T"] = _odd(rng, 16, min(65536, most))
        c["S"] = min(c["T"], _odd(rng, 1, 32))
    else:
        c["S"] = _odd(rng, 1, 16)
        c["T"] = c["S"] * _odd(rng, 1, max(1, min(16384, most // c["S"])))
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
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    T, D, way = case["T"], case["D"], case["way"]
    dt = DT[case["dtype"]]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=g, device=dev) * (hi - lo) + lo

    s = dict(case=case)
    if case["op"] == "norm":
        rt = DT[case["res"]]
        s["x"] = normal(T, D)
        s["gate"] = normal(T, D) if case["gate"] else None
        s["w_post"] = uniform(D, lo=0.5, hi=1.5).to(dt) if case["post"] else None
        s["b_post"] = normal(D, std=0.1) if case["post"] and case["kind"] == "layer" else None
        s["scale"] = uniform(D, lo=0.1, hi=1.0).to(dt) if case["scale"] else None
        s["res"] = normal(T, D, std=2.0, dtype=rt)
        s["w_pre"] = uniform(D, lo=0.5, hi=1.5).to(dt) if case["pre"] else None
        s["b_pre"] = normal(D, std=0.1) if case["pre"] and case["kind"] == "layer" else None
        if way == "train":
            s["dy"] = normal(T, D) if case["pre"] else None
            s["dres_out"] = normal(T, D, dtype=rt)
        if own:
            _own_norm(s)
        return s

    lens = lengths(case)
    s["lens"] = lens
    s["starts"] = None
    if case["ragged"]:
        s["starts"] = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=dev)
    S = case["S"]
    if case["op"] == "conv":
        W = case["W"]
        s["x"] = normal(T, 2 * D)[:, :D]              # the first half of a projection to 2 D channels
        s["w"] = ((uniform(D, W) * 2 - 1) / math.sqrt(W)).to(dt)
        s["bias"] = ((uniform(D) * 2 - 1) / math.sqrt(W)).to(dt)
        s["state"] = normal(S, W - 1, D) if way != "train" else None
        if way == "train":
            s["dy"] = normal(T, D)
        if own:
            _own_conv(s)
        return s

    N, G = case["N"], case["G"]
    a = normal(T, D, dtype=torch.float32)
    s["x"] = (a / (1 + torch.exp(-a))).to(dt)         # what the convolution's silu leaves
    s["z"] = normal(T, 2 * D)[:, D:]
    R = max(1, D // 16)
    p = normal(T, R + 2 * G * N)                      # the projection that holds dt's rank, B and C
    s["B"], s["C"] = p[:, R:R + G * N], p[:, R + G * N:]
    s["dt"] = normal(T, D, std=0.5)
    step = torch.exp(uniform(D, lo=math.log(1e-3), hi=math.log(1e-1)))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["A"] = -(torch.arange(1, N + 1, device=dev).float().expand(D, N) * uniform(D, 1, lo=0.8, hi=1.2)).contiguous()
    s["D"] = uniform(D, lo=0.5, hi=1.5)
    s["h"] = normal(S, D, N, std=0.2, dtype=torch.float32) if way != "train" else None
    if way == "train":
        s["dy"] = normal(T, D)
    if own:
        _own_scan(s)
    return s


# ----------------------------------------------------------------------- the library's own calls
def _codes(case):
    from convolution_forward_implicit_gb300 import seq
    from convolution_forward_implicit_gb300.binding import CONV_BF16, CONV_F32
    code = {"bf16": CONV_BF16, "f32": CONV_F32}
    return seq, code[case["dtype"]], code[case.get("res", "f32")]


def _own_conv(s):
    c = s["case"]
    seq, code, _ = _codes(c)
    S, T, D, W = c["S"], c["T"], c["D"], c["W"]
    kw = dict(ragged=c["ragged"])
    e = lambda *shape, dtype=s["x"].dtype: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    s["plan"] = seq.SeqConvPlan(S, T, D, W, code, "step" if c["way"] == "step" else "fwd", **kw).allocate()
    s["y"] = e(T, D)
    if c["way"] == "train":
        s["bwd"] = seq.SeqConvPlan(S, T, D, W, code, "bwd", **kw).allocate()
        s["dx"], s["dw"], s["dbias"] = e(T, D), e(D, W, dtype=torch.float32), e(D, dtype=torch.float32)
    else:
        s["state_out"] = e(S, W - 1, D)


def _own_scan(s):
    c = s["case"]
    seq, code, _ = _codes(c)
    S, T, D, N, G = c["S"], c["T"], c["D"], c["N"], c["G"]
    kw = dict(G=G, ragged=c["ragged"])
    f32 = torch.float32
    e = lambda *shape, dtype=s["x"].dtype: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    s["plan"] = seq.SeqScanPlan(S, T, D, N, code, "step" if c["way"] == "step" else "fwd", **kw).allocate()
    s["y"] = e(T, D)
    if c["way"] == "train":
        s["bwd"] = seq.SeqScanPlan(S, T, D, N, code, "bwd", **kw).allocate()
        s["saved"] = s["bwd"].allocate_saved()
        s["dx"], s["ddt"], s["dz"], s["dB"], s["dC"] = e(T, D), e(T, D), e(T, D), e(T, G * N), e(T, G * N)
        s["dA"], s["dD"], s["ddt_bias"] = e(D, N, dtype=f32), e(D, dtype=f32), e(D, dtype=f32)
    else:
        s["h_out"] = e(S, D, N, dtype=f32)


def _own_norm(s):
    c = s["case"]
    seq, code, res = _codes(c)
    T, D = c["T"], c["D"]
    kw = dict(res_dtype=res, kind=seq.SEQ_NORM_RMS if c["kind"] == "rms" else seq.SEQ_NORM_LAYER, post=c["post"],
              pre=c["pre"], gate=seq.SEQ_GATE_BEFORE if c["gate"] else seq.SEQ_GATE_NONE, residual=True, eps=1e-5)
    like = lambda t: None if t is None else torch.empty_like(t)  # noqa: E731
    s["plan"] = seq.SeqNormPlan(T, D, code, "fwd", **kw).allocate()
    s["y"], s["res_out"] = like(s["x"]) if c["pre"] else None, like(s["res"])
    if c["way"] == "train":
        s["bwd"] = seq.SeqNormPlan(T, D, code, "bwd", **kw).allocate()
        s["dx"], s["dgate"], s["dres"] = like(s["x"]), like(s["gate"]), like(s["res"])
        for k in ("w_post", "b_post", "scale", "w_pre", "b_pre"):
            s["d" + k] = None if s[k] is None else torch.empty(D, device="cuda")


def _run_own(s):
    c = s["case"]
    if c["op"] == "conv":
        x, w, b, st = s["x"], s["w"], s["bias"], s["starts"]
        if c["way"] == "step":
            s["plan"].step(x, w, b, s["state"], s["state_out"], s["y"])
            return {"y": s["y"], "state": s["state_out"]}
        if c["way"] == "prompt":
            s["plan"].forward(x, w, b, s["y"], starts=st, state_in=s["state"], state_out=s["state_out"])
            return {"y": s["y"], "state": s["state_out"]}
        s["plan"].forward(x, w, b, s["y"], starts=st)
        s["bwd"].backward(x, w, b, s["dy"], s["dx"], s["dw"], s["dbias"], starts=st)
        return {k: s[k] for k in ("y", "dx", "dw", "dbias")}
    if c["op"] == "scan":
        a = (s["x"], s["dt"], s["A"], s["B"], s["C"])
        kw = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
        if c["way"] == "step":
            s["plan"].step(*a, s["h"], s["h_out"], s["y"], **kw)
            return {"y": s["y"], "h": s["h_out"]}
        if c["way"] == "prompt":
            s["plan"].forward(*a, s["y"], starts=s["starts"], h_in=s["h"], h_out=s["h_out"], **kw)
            return {"y": s["y"], "h": s["h_out"]}
        s["plan"].forward(*a, s["y"], starts=s["starts"], saved=s["saved"], **kw)
        s["bwd"].backward(*a, s["dy"], s["saved"], s["dx"], s["ddt"], s["dA"], s["dB"], s["dC"], starts=s["starts"],
                          dD=s["dD"], dz=s["dz"], ddt_bias=s["ddt_bias"], **kw)
        return {k: s[k] for k in ("y", "dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias")}
    w = {k: s[k] for k in ("gate", "w_post", "b_post", "scale", "res", "w_pre", "b_pre")}
    s["plan"].forward(s["x"], y=s["y"], res_out=s["res_out"], **w)
    out = {"y": s["y"], "res_out": s["res_out"]}
    if c["way"] == "train":
        grads = {k: s[k] for k in ("dx", "dgate", "dw_post", "db_post", "dscale", "dres", "dw_pre", "db_pre")}
        s["bwd"].backward(s["x"], dy=s["dy"], dres_out=s["dres_out"], **grads, **w)
        out.update(grads)
    return out


# ----------------------------------------------------------------------------- the plain forms
def _silu(v):
    return v / (1 + torch.exp(-v))


def _dsilu(v):
    sig = 1 / (1 + torch.exp(-v))
    return sig * (1 + v * (1 - sig))


def _ends(lens, dev):
    """Indices of the sequences that hold tokens, their first and their last tokens."""
    n = torch.tensor(lens, device=dev)
    end = n.cumsum(0)
    full = (n > 0).nonzero()[:, 0]
    return n, full, (end - n)[full], end[full] - 1


def _plain_conv(s):
    c = s["case"]
    W, dt = c["W"], s["x"].dtype
    x, w, b = s["x"].float(), s["w"].float(), s["bias"].float()
    state = s["state"].float() if s["state"] is not None else x.new_zeros(c["S"], W - 1, c["D"])
    if c["way"] == "step":
        win = torch.cat([state, x[:, None]], 1)                       # S, W, D
        pre = (win * w.t()).sum(1) + b
        return {"y": _silu(pre).to(dt), "state": win[:, 1:].to(dt)}
    # every token's window as rows of [its sequence's state; its sequence's tokens]
    n, full, first, last = _ends(s["lens"], x.device)
    seq = torch.repeat_interleave(torch.arange(c["S"], device=x.device), n)
    begin = (n.cumsum(0) - n)[seq]
    T = c["T"]
    src = torch.arange(T, device=x.device)[:, None] + torch.arange(1 - W, 1, device=x.device)   # T, W
    back = src - begin[:, None]                                       # position in the sequence
    flat = torch.cat([x, state.reshape(-1, c["D"])])
    row = torch.where(back >= 0, src, T + seq[:, None] * (W - 1) + back + W - 1)
    win = flat[row]                                                   # T, W, D
    pre = (win * w.t()).sum(1) + b
    out = {"y": _silu(pre).to(dt)}
    if c["way"] == "prompt":
        pos = n[:, None] + torch.arange(1 - W, 0, device=x.device)    # S, W-1 positions in the sequence
        row = torch.where(pos >= 0, (n.cumsum(0) - n)[:, None] + pos,
                          T + torch.arange(c["S"], device=x.device)[:, None] * (W - 1) + pos + W - 1)
        out["state"] = flat[row].to(dt)
        return out
    dpre = s["dy"].float() * _dsilu(pre)
    out["dw"] = (dpre[:, None] * win).sum(0).t().contiguous()
    out["dbias"] = dpre.sum(0)
    stop = n.cumsum(0)[seq]
    dst = torch.arange(T, device=x.device)[:, None] + torch.arange(W, device=x.device)          # T, W: token t+i uses x[t] at tap W-1-i
    padded = torch.cat([dpre, dpre.new_zeros(1, c["D"])])
    grads = padded[torch.where(dst < stop[:, None], dst, T)]
    out["dx"] = (grads * w.t().flip(0)).sum(1).to(dt)
    return out


def _scan(a, b, most):
    """In place, b_t + a_t b_{t-1} + a_t a_{t-1} b_{t-2} + ... along the first axis, by doubling:
    after a pass with k each entry holds its last 2k terms; `most` terms are enough."""
    k = 1
    while k < most:
        b[k:] = b[k:] + a[k:] * b[:-k]
        a[k:] = a[k:] * a[:-k]
        k *= 2
    return b


def _plain_scan(s):
    c = s["case"]
    dt, G, N, D, T, S = s["x"].dtype, c["G"], c["N"], c["D"], c["T"], c["S"]
    x, z = s["x"].float(), s["z"].float()
    wide = lambda m: m.float().reshape(T, G, 1, N).expand(T, G, D // G, N).reshape(T, D, N)  # noqa: E731
    raw = s["dt"].float() + s["dt_bias"]
    delta = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    u = delta * x
    e = torch.exp(delta[:, :, None] * s["A"])
    Bw, Cw = wide(s["B"]), wide(s["C"])
    if c["way"] == "step":
        h = e * s["h"] + u[:, :, None] * Bw
        y = ((h * Cw).sum(-1) + s["D"] * x) * _silu(z)
        return {"y": y.to(dt), "h": h}
    n, full, first, last = _ends(s["lens"], x.device)
    most = max(s["lens"])
    a, h = e.clone(), u[:, :, None] * Bw
    if s["h"] is not None:
        h[first] += a[first] * s["h"][full]
    a[first] = 0
    h = _scan(a, h, most)
    core = (h * Cw).sum(-1) + s["D"] * x
    gz = _silu(z)
    out = {"y": (core * gz).to(dt)}
    if c["way"] == "prompt":
        hn = s["h"].clone()
        hn[full] = h[last]
        out["h"] = hn
        return out
    dout = s["dy"].float()
    dyc = dout * gz
    out["dz"] = (dout * core * _dsilu(z)).to(dt)
    nxt = e.roll(-1, 0)                                              # a_{t+1}
    nxt[last] = 0
    g = _scan(nxt.flip(0), (dyc[:, :, None] * Cw).flip(0), most).flip(0)
    before = h.roll(1, 0)
    before[first] = 0
    q = g * e * before                                               # dL/d(delta A)
    gB = (g * Bw).sum(-1)
    ddelta = (q * s["A"]).sum(-1) + x * gB
    out["dx"] = (delta * gB + s["D"] * dyc).to(dt)
    draw = ddelta / (1 + torch.exp(-raw))
    out["ddt"], out["ddt_bias"] = draw.to(dt), draw.sum(0)
    out["dA"] = (q * delta[:, :, None]).sum(0)
    out["dD"] = (dyc * x).sum(0)
    per = lambda m: m.reshape(T, G, D // G, N).sum(2).reshape(T, G * N).to(dt)  # noqa: E731
    out["dB"] = per(g * u[:, :, None])
    out["dC"] = per(h * dyc[:, :, None])
    return out


def _normed(v, layer, eps=1e-5):
    if layer:
        v = v - v.mean(1, keepdim=True)
    r = torch.rsqrt((v * v).mean(1, keepdim=True) + eps)
    return v * r, r


def _back(d, hat, r, layer):
    d = d - hat * (d * hat).mean(1, keepdim=True) - (d.mean(1, keepdim=True) if layer else 0)
    return d * r


def _plain_norm(s):
    c = s["case"]
    layer, dt, rt = c["kind"] == "layer", s["x"].dtype, s["res"].dtype
    f = {k: v.float() for k, v in s.items() if isinstance(v, torch.Tensor)}
    v = f["x"] * _silu(f["gate"]) if c["gate"] else f["x"]
    u = v
    if c["post"]:
        hat, ru = _normed(v, layer)
        u = hat * f["w_post"] + f.get("b_post", 0)
    r = f["res"] + u * f.get("scale", 1)
    out = {"res_out": r.to(rt), "y": None}
    if c["pre"]:
        hat2, rr = _normed(r, layer)
        out["y"] = (hat2 * f["w_pre"] + f.get("b_pre", 0)).to(dt)
    if c["way"] == "step":
        return out
    out.update({k: None for k in ("dx", "dgate", "dw_post", "db_post", "dscale", "dres", "dw_pre", "db_pre")})
    d = f["dres_out"]
    if c["pre"]:
        out["dw_pre"] = (f["dy"] * hat2).sum(0)
        if layer:
            out["db_pre"] = f["dy"].sum(0)
        d = d + _back(f["dy"] * f["w_pre"], hat2, rr, layer)
    out["dres"] = d.to(rt)
    if c["scale"]:
        out["dscale"] = (d * u).sum(0)
        d = d * f["scale"]
    if c["post"]:
        out["dw_post"] = (d * hat).sum(0)
        if layer:
            out["db_post"] = d.sum(0)
        d = _back(d * f["w_post"], hat, ru, layer)
    if c["gate"]:
        out["dgate"] = (d * f["x"] * _dsilu(f["gate"])).to(dt)
        d = d * _silu(f["gate"])
    out["dx"] = d.to(dt)
    return out


def run(state):
    if own:
        return _run_own(state)
    return {"conv": _plain_conv, "scan": _plain_scan, "norm": _plain_norm}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------ the floor
def work(case):
    T, D, way = case["T"], case["D"], case["way"]
    e = 2 if case["dtype"] == "bf16" else 4
    n = T * D
    if case["op"] == "norm":
        r = 2 if case["res"] == "bf16" else 4
        fwd = n * (e + r + r + (e if case["gate"] else 0) + (e if case["pre"] else 0))
        ops = n * (8 + 6 * case["post"] + 6 * case["gate"])
        if way == "step":
            return {"bytes": fwd, "flops": ops}
        return {"bytes": fwd + n * (e + r + r + (e if case["gate"] else 0) + (e if case["pre"] else 0)), "flops": 4 * ops}
    if case["op"] == "conv":
        W, S = case["W"], case["S"]
        if way == "train":
            return {"bytes": 4 * n * e + 2 * D * W * e, "flops": n * (6 * W + 20)}
        return {"bytes": 2 * n * e + 2 * S * (W - 1) * D * e + D * W * e, "flops": n * (2 * W + 6)}
    N, G, S = case["N"], case["G"], case["S"]
    if way == "train":
        return {"bytes": 8 * n * e + 4 * T * G * N * e + 8 * D * N, "flops": n * (22 * N + 40)}
    return {"bytes": 4 * n * e + 2 * T * G * N * e + 8 * S * D * N + 4 * D * N, "flops": n * (7 * N + 20)}


# ------------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    """The definitions, token by token in 64 bits; gradients by differentiating them."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    train = case["way"] == "train"
    names = {"conv": ("x", "w", "bias"), "scan": ("x", "dt", "A", "B", "C", "D", "z", "dt_bias"),
             "norm": ("x", "gate", "w_post", "b_post", "scale", "res", "w_pre", "b_pre")}[case["op"]]
    v = {k: (t.double().detach().requires_grad_(train) if isinstance(t, torch.Tensor) and t.is_floating_point() else t)
         for k, t in s.items()}
    with torch.set_grad_enabled(train):
        out = {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm}[case["op"]](case, v)
    if train:
        loss = 0
        if out.get("y") is not None:
            loss = loss + (out["y"] * v["dy"].detach()).sum()
        if case["op"] == "norm":
            loss = loss + (out["res_out"] * v["dres_out"].detach()).sum()
        have = [k for k in names if v[k] is not None]
        grads = torch.autograd.grad(loss, [v[k] for k in have])
        for k in names:
            out["d" + k] = None
        out.update({"d" + k: g for k, g in zip(have, grads)})
    return {k: t if t is None else t.detach() for k, t in out.items()}


def _exact_conv(case, v):
    W, ys, states = case["W"], [], []
    t = 0
    for i, n in enumerate(lengths(case)):
        head = v["state"][i] if v["state"] is not None else v["x"].new_zeros(W - 1, case["D"])
        full = torch.cat([head, v["x"][t:t + n]])
        pre = v["bias"].expand(n, -1)
        for j in range(W):
            pre = pre + v["w"][:, j] * full[j:j + n]
        ys.append(pre * torch.sigmoid(pre))
        states.append(full[n:])
        t += n
    out = {"y": torch.cat(ys)}
    if case["way"] != "train":
        out["state"] = torch.stack(states)
    return out


def _exact_scan(case, v):
    """All sequences advance together, longest first, so that those still running are a prefix."""
    lens = lengths(case)
    S, T, D, N, G = (case[k] for k in ("S", "T", "D", "N", "G"))
    dev = v["x"].device
    order = sorted(range(S), key=lambda i: -lens[i])
    begin = [sum(lens[:i]) for i in range(S)]
    delta = torch.nn.functional.softplus(v["dt"] + v["dt_bias"], threshold=1e9)
    B, C = v["B"].reshape(T, G, N), v["C"].reshape(T, G, N)
    h = v["h"][order].reshape(S, G, D // G, N) if v["h"] is not None else v["x"].new_zeros(S, G, D // G, N)
    A = v["A"].reshape(G, D // G, N)
    at = torch.tensor([begin[i] for i in order], device=dev)
    done, rows, ys, m = [], [], [], S
    for t in range(max(lens)):
        while m and lens[order[m - 1]] <= t:
            m -= 1
        done.append(h[m:])
        h = h[:m]
        row = at[:m] + t
        d = delta[row].reshape(m, G, D // G, 1)
        h = torch.exp(d * A) * h + d * v["x"][row].reshape(m, G, D // G, 1) * B[row][:, :, None]
        ys.append((h * C[row][:, :, None]).sum(-1).reshape(m, D))
        rows.append(row)
    done.append(h)
    back = torch.empty(T, dtype=torch.long, device=dev)
    back[torch.cat(rows)] = torch.arange(T, device=dev)
    y = torch.cat(ys)[back] + v["D"] * v["x"]
    out = {"y": y * v["z"] * torch.sigmoid(v["z"])}
    if case["way"] != "train":
        # sequences left in reverse order of their place in `order`
        hn = torch.cat(done[::-1]).reshape(S, D, N)
        out["h"] = torch.empty_like(hn)
        out["h"][torch.tensor(order, device=dev)] = hn
    return out


def _exact_norm(case, v):
    def norm(a, w, b):
        if case["kind"] == "layer":
            a = a - a.mean(1, keepdim=True)
        a = a / torch.sqrt(a.square().mean(1, keepdim=True) + 1e-5) * w
        return a if b is None else a + b

    u = v["x"] if v["gate"] is None else v["x"] * (v["gate"] * torch.sigmoid(v["gate"]))
    if case["post"]:
        u = norm(u, v["w_post"], v["b_post"])
    if case["scale"]:
        u = u * v["scale"]
    r = v["res"] + u
    return {"y": norm(r, v["w_pre"], v["b_pre"]) if case["pre"] else None, "res_out": r}
