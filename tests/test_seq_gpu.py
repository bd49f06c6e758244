"""The sequence-mixing operators on the GPU against the 64-bit oracle, element by element, within
bounds counted from their operations (tests/seq_oracle.py): sizes, strides, sequence lengths and
states where they can go wrong, both types, every direction."""
import numpy as np
import pytest

from convolution_forward_implicit_gb300 import seq as Q
from convolution_forward_implicit_gb300.binding import CONV_BF16, CONV_F32
from tests import seq_oracle as O

pytestmark = pytest.mark.gpu
SENTINEL = -12288.0


class Box:
    """Device tensors of one case: rounded inputs with their exact values, outputs between guards."""

    def __init__(self, seed, bf16):
        import torch
        self.rng = np.random.default_rng(seed)
        self.bf16 = bf16
        self.t = torch.bfloat16 if bf16 else torch.float32
        self.guards = []

    def put(self, a, dtype=None, pad=0, shift=0):
        """The values as a device tensor (rows with `pad` further columns, starting `shift` elements
        behind an aligned address) and their exact 64-bit values."""
        import torch
        dtype = dtype or self.t
        v = torch.from_numpy(np.asarray(a, dtype=np.float32)).to(dtype)
        exact = v.double().numpy()
        if pad or shift:
            cols = v.shape[-1] + pad
            flat = torch.full((v.shape[0] * cols + shift + 8,), SENTINEL, dtype=dtype, device="cuda")
            d = flat[shift:shift + v.shape[0] * cols].view(v.shape[0], cols)[:, :v.shape[-1]]
            d.copy_(v)
            return d, exact
        return v.cuda(), exact

    def normal(self, *shape, std=1.0, **kw):
        return self.put(self.rng.standard_normal(shape) * std, **kw)

    def out(self, *shape, dtype=None, pad=0):
        import torch
        dtype = dtype or self.t
        cols = shape[-1] + pad
        n = int(np.prod(shape[:-1], dtype=np.int64)) * cols
        buf = torch.full((n + 128,), SENTINEL, dtype=dtype, device="cuda")
        full = buf[64:64 + n].view(*shape[:-1], cols)
        self.guards.append((buf, n, full, shape[-1]))
        return full[..., :shape[-1]]

    def check_guards(self):
        for buf, n, full, width in self.guards:
            assert bool((buf[:64].float() == SENTINEL).all()) and bool((buf[64 + n:].float() == SENTINEL).all())
            assert bool((full[..., width:].float() == SENTINEL).all())


def host(t):
    return t.detach().double().cpu().numpy()


def starts_of(lens):
    import torch
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def slots_of(S, rng, count, drop=()):
    """A slot of its own for every sequence; those in `drop` get none."""
    import torch
    s = rng.permutation(count)[:S]
    s[list(drop)] = -1
    return s, torch.tensor(s, dtype=torch.int32, device="cuda")


UNIFORM = [[1], [7] * 3, [33], [300], [1] * 5, [16] * 2]
RAGGED = [[0, 1, 0, 0, 5, 2, 0], [3, 40, 1, 17], [0], [0, 0], [1, 1, 1, 1, 1, 1, 1, 1, 1], [129, 2, 64], [1, 0, 700, 3]]


# ------------------------------------------------------------------------------ convolution
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("lens,ragged", [(v, False) for v in UNIFORM] + [(v, True) for v in RAGGED])
@pytest.mark.parametrize("D,W,pad", [(16, 4, 0), (13, 3, 0), (264, 4, 8), (8, 1, 3), (24, 8, 0), (1, 2, 0)])
def test_conv(bf16, lens, ragged, D, W, pad):
    import torch
    S, T = len(lens), sum(lens)
    b = Box(17 * D + 3 * W + T, bf16)
    x, xe = b.normal(T, D, pad=pad)
    w, we = b.normal(D, W, std=W ** -0.5)
    bias, be = b.normal(D, std=0.3)
    dy, dye = b.normal(T, D, pad=pad)
    code = CONV_BF16 if bf16 else CONV_F32
    starts = starts_of(lens) if ragged else None
    # states: slots in any order, one sequence without a state
    state = state_out = sl = None
    se = np.zeros((S, W - 1, D))
    if W > 1:
        at, sl = slots_of(S, b.rng, S + 2, drop=[S // 2] if S > 2 else [])
        state, full = b.normal(S + 2, W - 1, D)
        se = np.where((at >= 0)[:, None, None], full[at], 0)
        state_out = b.out(S + 2, W - 1, D)
    y = b.out(T, D, pad=pad)
    p = Q.SeqConvPlan(S, T, D, W, code, ragged=ragged)
    p.forward(x, w, bias, y, starts=starts, state_in=state, state_out=state_out, slots=sl)
    ref, left, mag = O.conv(xe, we, be, lens, se)
    O.check("y", host(y), ref, mag, W + 100, bf16)
    if W > 1:
        got = host(state_out)
        for s in range(S):
            if at[s] >= 0:
                assert np.array_equal(got[at[s]], left[s])
        named = set(at[at >= 0])
        for r in range(S + 2):
            if r not in named:
                assert (got[r] == SENTINEL).all()
        # the same buffer for both states
        both = state.clone()
        p.forward(x, w, bias, y, starts=starts, state_in=both, state_out=both, slots=sl)
        O.check("y", host(y), ref, mag, W + 100, bf16)
        for s in range(S):
            if at[s] >= 0:
                assert np.array_equal(host(both)[at[s]], left[s])
    # gradients; no activation in half of the cases
    act = (D + W + S) % 2 == 0
    dx, dw, db = b.out(T, D, pad=pad), b.out(D, W, dtype=torch.float32), b.out(D, dtype=torch.float32)
    q = Q.SeqConvPlan(S, T, D, W, code, direction="bwd", ragged=ragged, silu=act)
    q.backward(x, w, bias, dy, dx, dw, db, starts=starts, state_in=state, slots=sl)
    ref, mag = O.conv_grad(xe, we, be, lens, se, dye, act=act)
    for name, v in (("dx", dx), ("dw", dw), ("dbias", db)):
        O.check(name, host(v), ref[name], mag[name], W + 100 + (0 if name == "dx" else T), bf16 and name == "dx")
    b.check_guards()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("S,D,W", [(1, 1, 2), (3, 40, 4), (5, 37, 3), (70, 8, 4), (2, 1032, 8), (4, 16, 1)])
def test_conv_step_continues_a_prompt(bf16, S, D, W):
    """Steps after a prompt give what the whole sequence gives."""
    L, more = 6, 3
    b = Box(S * D + W, bf16)
    code = CONV_BF16 if bf16 else CONV_F32
    x, xe = b.normal(S * (L + more), D)
    w, we = b.normal(D, W, std=W ** -0.5)
    bias, be = b.normal(D, std=0.3)
    ref, left, mag = O.conv(xe, we, be, [L + more] * S, np.zeros((S, W - 1, D)))
    x3, ref, mag = x.view(S, L + more, D), ref.reshape(S, -1, D), mag.reshape(S, -1, D)
    state = b.out(S, W - 1, D) if W > 1 else None
    y = b.out(S * L, D)
    Q.SeqConvPlan(S, S * L, D, W, code).forward(x3[:, :L].contiguous(), w, bias, y, state_out=state)
    O.check("prompt", host(y).reshape(S, L, D), ref[:, :L], mag[:, :L], W + 100, bf16)
    step = Q.SeqConvPlan(S, S, D, W, code, direction="step")
    for i in range(more):
        y1 = b.out(S, D)
        step.step(x3[:, L + i], w, bias, state, state, y1)      # rows L + more tokens apart
        O.check("step", host(y1), ref[:, L + i], mag[:, L + i], W + 100, bf16)
    if W > 1:
        assert np.array_equal(host(state), left)
    b.check_guards()


def test_conv_handles_unaligned_rows_and_extreme_inputs():
    b = Box(5, True)
    x, xe = b.normal(20, 64, shift=3, pad=5)
    w, we = b.normal(64, 4)
    big = xe.copy()
    big[3], big[7] = 3e4, -3e4
    x.copy_(b.put(big)[0])
    big = host(x)
    bias, be = b.normal(64)
    y = b.out(20, 64, pad=1)
    Q.SeqConvPlan(2, 20, 64, 4, CONV_BF16).forward(x, w, bias, y)
    ref, _, mag = O.conv(big, we, be, [10, 10], np.zeros((2, 3, 64)))
    O.check("y", host(y), ref, mag, 104, True)
    b.check_guards()


# ------------------------------------------------------------------------------------- scan
def scan_case(seed, bf16, lens, D, N, G, pad=0, z=True, skip=True, bias=True, act=True, states=True):
    import torch
    S, T = len(lens), sum(lens)
    b = Box(seed, bf16)
    f32 = torch.float32
    c = dict(S=S, T=T, D=D, N=N, G=G, act=act, box=b)
    dev, ex = {}, {}

    def put(name, pair):
        dev[name], ex[name] = pair

    put("x", b.normal(T, D, pad=pad))
    put("dt", b.put(b.rng.standard_normal((T, D)) * 0.7 + (-1 if act else 0), pad=pad))
    if not act:
        put("dt", b.put(b.rng.uniform(0.01, 0.7, (T, D)), pad=pad))
    put("A", b.put(-b.rng.uniform(0.2, 4, (D, N)), dtype=f32))
    put("B", b.normal(T, G * N, pad=pad))
    put("C", b.normal(T, G * N, pad=pad))
    if skip:
        put("D", b.normal(D, dtype=f32))
    if z:
        put("z", b.normal(T, D, std=2.0, pad=pad))
    if bias:
        put("dt_bias", b.normal(D, std=0.2, dtype=f32) if act else b.put(b.rng.uniform(0, 0.1, D), dtype=f32))
    c.update(dev=dev, ex=ex)
    c["at"], c["slots"], c["h"], he = None, None, None, np.zeros((S, D, N))
    if states:
        c["at"], c["slots"] = slots_of(S, b.rng, S + 1, drop=[S // 2] if S > 2 else [])
        c["h"], full = b.normal(S + 1, D, N, dtype=f32)
        he = np.where((c["at"] >= 0)[:, None, None], full[c["at"]], 0)
    c["he"] = he
    return c


def check_states(c, got, ref, mag, k, name):
    for s in range(c["S"]):
        if c["at"][s] >= 0:
            O.check(name, got[c["at"][s]], ref[s], mag[s], k, False)
    named = set(c["at"][c["at"] >= 0])
    for r in range(len(got)):
        if r not in named:
            assert (got[r] == SENTINEL).all()


SCANS = [  # D, N, G, pad, z, skip, bias, act
    (16, 16, 1, 0, 1, 1, 1, 1), (40, 16, 2, 8, 1, 1, 1, 1), (7, 1, 1, 0, 0, 0, 0, 1), (130, 5, 2, 3, 1, 0, 1, 0),
    (33, 24, 3, 0, 0, 1, 1, 1), (12, 64, 1, 0, 1, 1, 0, 1), (6, 128, 2, 1, 1, 1, 1, 1), (260, 8, 1, 0, 1, 1, 1, 1),
    (1, 16, 1, 0, 1, 1, 1, 0), (520, 4, 1, 8, 1, 1, 1, 1),
]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("lens,ragged", [(v, False) for v in UNIFORM] + [(v, True) for v in RAGGED])
@pytest.mark.parametrize("spec", SCANS)
def test_scan(bf16, lens, ragged, spec):
    import torch
    D, N, G, pad, z, skip, bias, act = spec
    S, T = len(lens), sum(lens)
    states = (D + T) % 3 != 0
    c = scan_case(31 * D + N + 7 * T, bf16, lens, D, N, G, pad, z, skip, bias, bool(act), states)
    b, dev, f32 = c["box"], c["dev"], torch.float32
    code = CONV_BF16 if bf16 else CONV_F32
    starts = starts_of(lens) if ragged else None
    dy, dye = b.normal(T, D, pad=pad)
    dh = dhe = None
    if states:
        dh, full = b.normal(S + 1, D, N, dtype=f32)
        dhe = np.where((c["at"] >= 0)[:, None, None], full[c["at"]], 0)
    ref, mag = O.scan(**c["ex"], G=G, lens=lens, h0=c["he"], act=bool(act), dy=dye, dh_out=dhe)
    k = 4 * max(lens, default=0) + N + 100
    arr = [dev.get(n) for n in ("x", "dt", "A", "B", "C")]
    opt = {n: dev.get(n) for n in ("D", "z", "dt_bias")}

    p = Q.SeqScanPlan(S, T, D, N, code, G=G, ragged=ragged, softplus=bool(act))
    q = Q.SeqScanPlan(S, T, D, N, code, direction="bwd", G=G, ragged=ragged, softplus=bool(act))
    assert p.saved_bytes == q.saved_bytes
    y, saved = b.out(T, D, pad=pad), q.allocate_saved()
    h_out = b.out(S + 1, D, N, dtype=f32) if states else None
    p.forward(*arr, y, **opt, starts=starts, h_in=c["h"], h_out=h_out, slots=c["slots"], saved=saved)
    O.check("y", host(y), ref["y"], mag["y"], k, bf16)
    if states:
        check_states(c, host(h_out), ref["h"], mag["h"], k, "h")

    dx, ddt, dz = (b.out(T, D, pad=pad) for _ in range(3))
    dB, dC = (b.out(T, G * N, pad=pad) for _ in range(2))
    dA, dD, ddb = b.out(D, N, dtype=f32), b.out(D, dtype=f32), b.out(D, dtype=f32)
    dh_in = b.out(S + 1, D, N, dtype=f32) if states else None
    q.backward(*arr, dy, saved, dx, ddt, dA, dB, dC, **opt, starts=starts, h_in=c["h"], dh_out=dh, dh_in=dh_in,
               slots=c["slots"], dz=dz if z else None, dD=dD if skip else None, ddt_bias=ddb if bias else None)
    got = dict(dx=(dx, 0), ddt=(ddt, 0), dB=(dB, D), dC=(dC, D), dA=(dA, T))
    got.update({n: (v, T) for n, v, on in (("dD", dD, skip), ("ddt_bias", ddb, bias)) if on})
    if z:
        got["dz"] = (dz, 0)
    for name, (v, more) in got.items():
        O.check(name, host(v), ref[name], mag[name], 2 * k + more, bf16 and v.dtype == torch.bfloat16)
    if states:
        check_states(c, host(dh_in), ref["dh_in"], mag["dh_in"], 2 * k, "dh_in")
        # the states may be left where they came from
        both = c["h"].clone()
        p.forward(*arr, y, **opt, starts=starts, h_in=both, h_out=both, slots=c["slots"])
        O.check("y", host(y), ref["y"], mag["y"], k, bf16)
        for s in range(S):
            if c["at"][s] >= 0:
                O.check("h in place", host(both)[c["at"][s]], ref["h"][s], mag["h"][s], k, False)
    b.check_guards()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("S,D,N,G", [(1, 16, 16, 1), (3, 70, 16, 2), (5, 9, 7, 1), (66, 8, 64, 1), (2, 140, 128, 1),
                                     (4, 33, 1, 3), (2, 24, 3, 1)])
def test_scan_step_continues_a_prompt(bf16, S, D, N, G):
    import torch
    L, more = 5, 3
    lens = [L + more] * S
    c = scan_case(S * D + N, bf16, lens, D, N, G, states=False)
    code = CONV_BF16 if bf16 else CONV_F32
    dev, b = c["dev"], c["box"]
    ref, mag = O.scan(**c["ex"], G=G, lens=lens, h0=np.zeros((S, D, N)))
    k = 4 * (L + more) + N + 100
    rows = {n: dev[n].view(S, L + more, -1) for n in ("x", "dt", "B", "C", "z")}
    head = {n: v[:, :L].contiguous() for n, v in rows.items()}
    h, y = b.out(S, D, N, dtype=torch.float32), b.out(S * L, D)
    Q.SeqScanPlan(S, S * L, D, N, code, G=G).forward(head["x"], head["dt"], dev["A"], head["B"], head["C"], y, D=dev["D"],
                                                     z=head["z"], dt_bias=dev["dt_bias"], h_out=h)
    yr, ym = ref["y"].reshape(S, -1, D), mag["y"].reshape(S, -1, D)
    O.check("prompt", host(y).reshape(S, L, D), yr[:, :L], ym[:, :L], k, bf16)
    step = Q.SeqScanPlan(S, S, D, N, code, direction="step", G=G)
    for i in range(more):
        t = {n: v[:, L + i] for n, v in rows.items()}           # rows L + more tokens apart
        y1 = b.out(S, D)
        step.step(t["x"], t["dt"], dev["A"], t["B"], t["C"], h, h, y1, D=dev["D"], z=t["z"], dt_bias=dev["dt_bias"])
        O.check("step", host(y1), yr[:, L + i], ym[:, L + i], k, bf16)
    O.check("h", host(h), ref["h"], mag["h"], k, False)
    b.check_guards()


def test_scan_step_with_slots():
    """Rows without a slot start from zero and leave nothing behind."""
    import torch
    S, D, N = 6, 20, 16
    c = scan_case(9, False, [1] * S, D, N, 1)
    dev = c["dev"]
    ref, mag = O.scan(**c["ex"], G=1, lens=[1] * S, h0=c["he"])
    h, y = c["box"].out(S + 1, D, N, dtype=torch.float32), c["box"].out(S, D)
    Q.SeqScanPlan(S, S, D, N, CONV_F32, direction="step").step(
        dev["x"], dev["dt"], dev["A"], dev["B"], dev["C"], c["h"], h, y, D=dev["D"], z=dev["z"], dt_bias=dev["dt_bias"],
        slots=c["slots"])
    O.check("y", host(y), ref["y"], mag["y"], 120, False)
    check_states(c, host(h), ref["h"], mag["h"], 120, "h")


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("lens,ragged", [([4100], False), ([2300, 2300], False), ([1, 900, 0, 2100, 33, 777, 8, 450], True),
                                         ([41 + i % 7 for i in range(100)], True)])
@pytest.mark.parametrize("spec", [(40, 16, 1, 0, 1, 1, 1, 1), (17, 5, 1, 1, 1, 1, 1, 1)])
def test_scan_in_many_pieces(bf16, lens, ragged, spec):
    """Few channels and a long axis: more pieces than one or four parts of the joining kernel take."""
    D, N, G = spec[:3]
    for direction in ("fwd", "bwd"):
        text = Q.SeqScanPlan(len(lens), sum(lens), D, N, CONV_BF16 if bf16 else CONV_F32, direction=direction, ragged=ragged).describe()
        assert 64 < int(text.split("pieces=")[1].split()[0])
    test_scan(bf16, lens, ragged, spec)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("S,D,N,G,pad", [(1300, 256, 16, 1, 0), (1301, 256, 16, 2, 8), (1301, 255, 16, 1, 0), (4901, 36, 24, 3, 0),
                                         (4900, 64, 7, 1, 0), (611, 24, 128, 1, 8)])
def test_scan_step_of_many_sequences(bf16, S, D, N, G, pad):
    """Several sequences, and where rows allow it two channels, to a thread; the last thread's may be fewer."""
    import torch
    c = scan_case(S + N, bf16, [1] * S, D, N, G, pad=pad)
    dev, b = c["dev"], c["box"]
    ref, mag = O.scan(**c["ex"], G=G, lens=[1] * S, h0=c["he"])
    h, y = b.out(S + 1, D, N, dtype=torch.float32), b.out(S, D, pad=pad)
    Q.SeqScanPlan(S, S, D, N, CONV_BF16 if bf16 else CONV_F32, direction="step", G=G).step(
        dev["x"], dev["dt"], dev["A"], dev["B"], dev["C"], c["h"], h, y, D=dev["D"], z=dev["z"], dt_bias=dev["dt_bias"],
        slots=c["slots"])
    O.check("y", host(y), ref["y"], mag["y"], N + 120, bf16)
    check_states(c, host(h), ref["h"], mag["h"], 120, "h")
    b.check_guards()


def test_scan_is_the_same_twice_and_on_another_stream():
    import torch
    lens = [700, 0, 1, 300]
    c = scan_case(11, True, lens, 136, 16, 1, states=False)
    dev = c["dev"]
    T = sum(lens)
    starts = starts_of(lens)
    p = Q.SeqScanPlan(4, T, 136, 16, CONV_BF16, ragged=True)
    ys = []
    for stream in (None, torch.cuda.Stream()):
        y = torch.empty(T, 136, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        p.forward(dev["x"], dev["dt"], dev["A"], dev["B"], dev["C"], y, starts=starts,
                  stream=None if stream is None else stream.cuda_stream)
        torch.cuda.synchronize()
        ys.append(y)
    assert torch.equal(*ys)


def test_scan_forward_in_a_graph():
    import torch
    c = scan_case(12, False, [40, 40], 24, 16, 1, states=False)
    dev = c["dev"]
    p = Q.SeqScanPlan(2, 80, 24, 16, CONV_F32).allocate()
    y, want = torch.empty(80, 24, device="cuda"), torch.empty(80, 24, device="cuda")
    args = [dev[n] for n in ("x", "dt", "A", "B", "C")]
    p.forward(*args, want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.forward(*args, y)
    y.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


# ------------------------------------------------------------------------------------- norm
@pytest.mark.parametrize("types", ["f32", "bf16", "bf16/f32"])
@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("rows,D,pad", [(1, 1, 0), (3, 8, 0), (5, 13, 2), (70, 384, 8), (2, 1288, 0), (9, 4096, 0),
                                        (3, 9001, 0), (2, 16384, 0), (611, 40, 0)])
@pytest.mark.parametrize("post,pre,gate,res,scale", [(0, 1, "none", 1, 0), (1, 1, "before", 1, 1), (1, 0, "after", 0, 0),
                                                     (1, 0, "none", 1, 1), (0, 1, "after", 0, 1), (1, 1, "after", 1, 1)])
def test_norm(types, layer, rows, D, pad, post, pre, gate, res, scale):
    import torch
    bf16 = types != "f32"
    rt = torch.bfloat16 if types == "bf16" else torch.float32
    b = Box(rows + D + 3 * post + pre, bf16)
    f32 = torch.float32
    code, rcode = CONV_BF16 if bf16 else CONV_F32, CONV_BF16 if types == "bf16" else CONV_F32
    eps = 1e-3
    dev, ex = {}, {}

    def put(name, on, pair):
        if on:
            dev[name], ex[name] = pair

    put("x", True, b.normal(rows, D, pad=pad))
    put("gate", gate != "none", b.normal(rows, D, std=2.0, pad=pad))
    put("w_post", post, b.put(b.rng.uniform(0.5, 1.5, D)))
    put("b_post", post and layer, b.normal(D, std=0.2))
    put("scale", scale, b.put(b.rng.uniform(0.1, 1, D)))
    put("res", res, b.put(b.rng.standard_normal((rows, D)) + 0.5, dtype=rt, pad=pad))
    put("w_pre", pre, b.put(b.rng.uniform(0.5, 1.5, D)))
    put("b_pre", pre and layer, b.normal(D, std=0.2))
    has_y = pre or not res
    dy, dye = b.normal(rows, D, pad=pad) if has_y else (None, None)
    dro, droe = b.normal(rows, D, dtype=rt, pad=pad) if res else (None, None)
    ref, mag = O.norm(**ex, layer=layer, eps=eps, post=post, pre=pre, after=gate == "after", dy=dye, dres_out=droe)
    kw = dict(res_dtype=rcode, kind="layer" if layer else "rms", post=bool(post), pre=bool(pre), gate=gate,
              residual=bool(res), eps=eps)
    y = b.out(rows, D, pad=pad) if has_y else None
    ro = b.out(rows, D, dtype=rt, pad=pad) if res else None
    others = {n: v for n, v in dev.items() if n != "x"}
    Q.SeqNormPlan(rows, D, code, **kw).forward(dev["x"], y=y, res_out=ro, **others)
    k = D ** 0.5 + 120        # a row's sums run over at most D / 32 + 10 values one after another
    k = max(k, D / 32 + 120)
    if has_y:
        O.check("y", host(y), ref["y"], mag["y"], k, bf16)
    if res:
        O.check("res_out", host(ro), ref["res_out"], mag["res_out"], k, rt == torch.bfloat16)
    grads = dict(dx=b.out(rows, D, pad=pad))
    if gate != "none":
        grads["dgate"] = b.out(rows, D, pad=pad)
    if res:
        grads["dres"] = b.out(rows, D, dtype=rt, pad=pad)
    for n in ("w_post", "b_post", "scale", "w_pre", "b_pre"):
        if n in dev:
            grads["d" + n] = b.out(D, dtype=f32)
    Q.SeqNormPlan(rows, D, code, direction="bwd", **kw).backward(dev["x"], dy=dy, dres_out=dro, **grads, **others)
    for n, v in grads.items():
        whole = v.dim() == 1
        O.check(n, host(v), ref[n], mag[n], 2 * k + (rows if whole else 0), v.dtype == torch.bfloat16)
    b.check_guards()


def test_norm_in_place_and_zero_rows():
    """The residual may be updated in place; a row of zeros normalises to the bias."""
    import torch
    b = Box(3, True)
    x, xe = b.normal(5, 64)
    r0, re_ = b.normal(5, 64, dtype=torch.float32)
    x[2], r0[2] = 0, 0
    xe[2], re_[2] = 0, 0
    w, we = b.normal(64)
    bias, be = b.normal(64)
    r = r0.clone()
    y = b.out(5, 64)
    Q.SeqNormPlan(5, 64, CONV_BF16, kind="layer").forward(x, y=y, res=r, res_out=r, w_pre=w, b_pre=bias)
    ref, mag = O.norm(xe, True, 1e-5, False, True, res=re_, w_pre=we, b_pre=be)
    O.check("y", host(y), ref["y"], mag["y"], 130, True)
    O.check("res", host(r), ref["res_out"], mag["res_out"], 130, False)
    assert np.array_equal(host(y)[2], be)


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("rows,D", [(5, 64), (3, 200), (2, 512)])
def test_norm_without_eps(rows, D, layer):
    """eps 0: rows that share a thread block with places behind the last row, which must add nothing."""
    import torch
    b = Box(rows + D, False)
    x, xe = b.normal(rows, D)
    r, re_ = b.normal(rows, D)
    w, we = b.put(b.rng.uniform(0.5, 1.5, D))
    wp, wpe = b.put(b.rng.uniform(0.5, 1.5, D))
    dy, dye = b.normal(rows, D)
    ref, mag = O.norm(xe, layer, 0.0, True, True, res=re_, w_post=wpe, w_pre=we, dy=dye)
    g = dict(dx=b.out(rows, D), dres=b.out(rows, D), dw_pre=b.out(D), dw_post=b.out(D))
    plan = Q.SeqNormPlan(rows, D, CONV_F32, direction="bwd", kind="layer" if layer else "rms", post=True, pre=True, eps=0.0)
    plan.backward(x, dy=dy, res=r, w_post=wp, w_pre=w, **g)
    k = 2 * max(D ** 0.5 + 120, D / 32 + 120)
    for n, v in g.items():
        O.check(n, host(v), ref[n], mag[n], k + (rows if v.dim() == 1 else 0), False)


def test_layer_norm_far_from_zero():
    """Whole numbers around 4096, and rows whose parts lie around different ones: their sums are exact in 24
    bits, so only the squares, the root and the last product round, about 40 times in a row in all."""
    import torch
    rng = np.random.default_rng(5)
    v = rng.integers(-8, 9, (6, 1024)).astype(np.float64) + 4096
    v[3:, 256:512] -= 64
    v[3:, 700:] += 32
    x = torch.from_numpy(v).float().cuda()
    y = torch.empty_like(x)
    Q.SeqNormPlan(6, 1024, CONV_F32, kind="layer", post=True, pre=False, residual=False, eps=0.0).forward(x, y=y)
    m = v - v.mean(1, keepdims=True)
    want = m / np.sqrt((m * m).mean(1, keepdims=True))
    assert np.all(np.abs(host(y) - want) <= 64 * 2.0 ** -24 * np.maximum(np.abs(want), 1))


# ---------------------------------------------------------------------------------- together
def test_block_example_decodes_what_the_whole_sequence_gives():
    """examples/ssm_block.py: a prompt and steps behind it against all tokens at once.  Between the calls
    every activation is rounded to bf16 (2^-9 relative); the two ways differ by such roundings only, over the
    handful of them that a token passes: far below 1e-2."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import ssm_block
    assert ssm_block.main(["--batch", "3", "--length", "40", "--width", "64", "--steps", "5"]) < 1e-2


@pytest.mark.parametrize("bf16,D", [(False, (1 << 22) - 3), (False, 1 << 22), (True, (1 << 22) - 3), (True, 2097121)])
def test_conv_gradients_of_the_widest_rows(bf16, D):
    """More blocks of channels than a launch's second dimension takes."""
    import torch
    lens, W = [2, 1], 2
    b = Box(D, bf16)
    x, xe = b.normal(3, D)
    w, we = b.normal(D, W)
    bias, be = b.normal(D, std=0.3)
    dy, dye = b.normal(3, D)
    dx, dw, db = b.out(3, D), b.out(D, W, dtype=torch.float32), b.out(D, dtype=torch.float32)
    Q.SeqConvPlan(2, 3, D, W, CONV_BF16 if bf16 else CONV_F32, direction="bwd", ragged=True).backward(
        x, w, bias, dy, dx, dw, db, starts=starts_of(lens))
    ref, mag = O.conv_grad(xe, we, be, lens, np.zeros((2, W - 1, D)), dye)
    for name, v in (("dx", dx), ("dw", dw), ("dbias", db)):
        O.check(name, host(v), ref[name], mag[name], W + 103, bf16 and name == "dx")
    b.check_guards()


@pytest.mark.parametrize("types", ["f32", "bf16", "bf16/f32"])
@pytest.mark.parametrize("rows,D,pad", [(1, 1, 0), (7, 13, 2), (9, 40, 0), (70, 384, 8), (700, 1288, 0), (9, 4096, 0), (700, 4096, 0), (3, 9001, 0),
                                        (2, 16384, 8)])
def test_norm_updates_the_residual_in_place(types, rows, D, pad):
    """res_out = res: the same bits as with a buffer of its own, behind the same rows, whatever else the call does."""
    import torch
    bf16, rt = types != "f32", torch.bfloat16 if types == "bf16" else torch.float32
    b = Box(rows + D, bf16)
    code, rcode = CONV_BF16 if bf16 else CONV_F32, CONV_BF16 if types == "bf16" else CONV_F32
    x, gate = b.normal(rows, D, pad=pad)[0], b.normal(rows, D, pad=pad)[0]
    w = {k: b.normal(D)[0] for k in ("w_post", "b_post", "scale", "w_pre", "b_pre")}
    res = b.out(rows, D, dtype=rt, pad=pad)
    first = b.put(b.rng.standard_normal((rows, D)), dtype=rt)[0]
    for kind in ("rms", "layer"):
        for post, pre in ((True, True), (False, True), (True, False)):
            p = Q.SeqNormPlan(rows, D, code, res_dtype=rcode, kind=kind, post=post, pre=pre, gate="before")
            args = {k: v for k, v in w.items() if not (k.endswith("post") and not post) and not (k.endswith("pre") and not pre)}
            res.copy_(first)
            y, ro = (b.out(rows, D, pad=pad) if pre else None), b.out(rows, D, dtype=rt, pad=pad)
            p.forward(x, y=y, gate=gate, res=res, res_out=ro, **args)
            y2 = b.out(rows, D, pad=pad) if pre else None
            p.forward(x, y=y2, gate=gate, res=res, res_out=res, **args)
            assert torch.equal(res, ro) and (not pre or torch.equal(y, y2))
    b.check_guards()


LONG = [([600], False), ([1300], False), ([300, 1200], True), ([4100], False), ([2300, 2300], False), ([1, 900, 0, 2100, 33, 777, 8, 450], True)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("lens,ragged", LONG)
@pytest.mark.parametrize("D,N,pad", [(40, 16, 0), (17, 5, 1)])
def test_scan_of_long_memory(bf16, lens, ragged, D, N, pad):
    """States that keep half of what they held through every part of the pieces' joining, and inputs that are zero in
    most tokens: outputs, states and gradients come a long way (wrong joins leave these bounds, see the host tests)."""
    import torch
    S, T, f32 = len(lens), sum(lens), torch.float32
    b = Box(T + D, bf16)
    a, more = O.slow_case(b.rng, lens, D, N)
    dev, ex = {}, {}
    for name, v in a.items():
        one = name in ("A", "D")
        dev[name], ex[name] = b.put(v, dtype=f32 if one else None, pad=0 if one else pad)
    h, he = b.put(more["h"], dtype=f32)
    dh, dhe = b.put(more["dh"], dtype=f32)
    dy, dye = b.put(more["dy"], pad=pad)
    ref, mag = O.scan(**ex, G=1, lens=lens, h0=he, dy=dye, dh_out=dhe)
    k = 4 * max(lens) + N + 100
    code, starts = CONV_BF16 if bf16 else CONV_F32, starts_of(lens) if ragged else None
    arr = [dev[n] for n in ("x", "dt", "A", "B", "C")]
    p, q = (Q.SeqScanPlan(S, T, D, N, code, direction=d, ragged=ragged) for d in ("fwd", "bwd"))
    for plan in (p, q):
        pieces = int(plan.describe().split("pieces=")[1].split()[0])
        assert 16 < pieces / (1 if ragged else S) <= 128
    y, saved, left = b.out(T, D, pad=pad), q.allocate_saved(), b.out(S, D, N, dtype=f32)
    p.forward(*arr, y, D=dev["D"], starts=starts, h_in=h, h_out=left, saved=saved)
    O.check("y", host(y), ref["y"], mag["y"], k, bf16)
    O.check("h", host(left), ref["h"], mag["h"], k, False)
    out = dict(dx=(T, D), ddt=(T, D), dA=(D, N), dB=(T, N), dC=(T, N), dD=(D,), dh_in=(S, D, N))
    g = {n: b.out(*s, dtype=f32 if n in ("dA", "dD", "dh_in") else None, pad=pad if n in ("dx", "ddt", "dB", "dC") else 0) for n, s in out.items()}
    q.backward(*arr, dy, saved, D=dev["D"], starts=starts, h_in=h, dh_out=dh, **g)
    for n, v in g.items():
        O.check(n, host(v), ref[n], mag[n], 2 * k + (T if n in ("dA", "dD") else D if n in ("dB", "dC") else 0), v.dtype == torch.bfloat16)
    b.check_guards()


# --------------------------------------------------------------------------------- rounding
def test_bf16_outputs_are_rounded_to_nearest_even():
    """Sums of two bf16 numbers on one grid of 2^-7 and products of two are exact in fp32: what is written is them
    rounded once, many of the sums halfway between two bf16 numbers."""
    import torch
    rng = np.random.default_rng(6)
    T, D = 96, 72
    grid = lambda *s: torch.from_numpy(rng.integers(-255, 256, s).astype(np.float32) * 2.0 ** -7)      # noqa: E731
    bf = lambda t: t.to(torch.bfloat16)      # noqa: E731   (nearest, ties to even)
    gpu = lambda t: bf(t).cuda()      # noqa: E731
    out = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device="cuda")      # noqa: E731
    x, r, dy = grid(T, D), grid(T, D), grid(T, D)
    late = lambda v: torch.cat([v[1:], torch.zeros(1, D)])      # noqa: E731
    early = lambda v: torch.cat([torch.zeros(1, D), v[:-1]])      # noqa: E731
    ties = (bf(x + early(x)).float() != x + early(x)).float().mean()
    assert ties > 0.1
    # convolution with taps of one, without activation: forward, gradient, steps
    w = torch.ones(D, 2)
    y, dx = out(T, D), out(T, D)
    Q.SeqConvPlan(1, T, D, 2, CONV_BF16, silu=False).forward(gpu(x), gpu(w), None, y)
    assert torch.equal(y.cpu(), bf(x + early(x)))
    q = Q.SeqConvPlan(1, T, D, 2, CONV_BF16, direction="bwd", silu=False)
    q.backward(gpu(x), gpu(w), None, gpu(dy), dx, out(D, 2, dtype=torch.float32), None)
    assert torch.equal(dx.cpu(), bf(dy + late(dy)))
    state = gpu(r).view(T, 1, D)
    Q.SeqConvPlan(T, T, D, 2, CONV_BF16, direction="step", silu=False).step(gpu(x), gpu(w), None, state, state, y)
    assert torch.equal(y.cpu(), bf(x + r)) and torch.equal(state.cpu().view(T, D), bf(x))
    # the residual
    ro = out(T, D)
    Q.SeqNormPlan(T, D, CONV_BF16, res_dtype=CONV_BF16).forward(gpu(x), y=y, res=gpu(r), res_out=ro)
    assert torch.equal(ro.cpu(), bf(x + r))
    # scan with steps of zero and no states: the skip connection alone, y = D x and dx = D dy
    Dv = torch.from_numpy(rng.integers(129, 256, D).astype(np.float32) * 2.0 ** -7)
    zero = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    A, B = -torch.ones(D, 16, device="cuda"), gpu(grid(T, 16))
    for S in (1, 12):
        p, q = (Q.SeqScanPlan(S, T, D, 16, CONV_BF16, direction=d, softplus=False) for d in ("fwd", "bwd"))
        saved = q.allocate_saved()
        p.forward(gpu(x), zero, A, B, B, y, D=Dv.cuda(), saved=saved)
        assert torch.equal(y.cpu(), bf(Dv * x))
        q.backward(gpu(x), zero, A, B, B, gpu(dy), saved, dx, out(T, D), out(D, 16, dtype=torch.float32), out(T, 16), out(T, 16), D=Dv.cuda(),
                   dD=out(D, dtype=torch.float32))
        assert torch.equal(dx.cpu(), bf(Dv * dy))
    h = torch.zeros(T, D, 16, device="cuda")
    Q.SeqScanPlan(T, T, D, 16, CONV_BF16, direction="step", softplus=False).step(gpu(x), zero, A, B, B, h, h, y, D=Dv.cuda())
    assert torch.equal(y.cpu(), bf(Dv * x))


# ----------------------------------------------------------------------- one column, bad values
@pytest.mark.parametrize("types", ["f32", "bf16", "bf16/f32"])
@pytest.mark.parametrize("rows", [1, 5, 611])
def test_layer_norm_of_one_column(types, rows):
    """A column less its mean is zero: what is behind the norm is its bias, and nothing of a gradient passes it."""
    import torch
    bf16, rt = types != "f32", torch.bfloat16 if types == "bf16" else torch.float32
    b = Box(rows, bf16)
    f32 = torch.float32
    code, rcode = CONV_BF16 if bf16 else CONV_F32, CONV_BF16 if types == "bf16" else CONV_F32
    x = b.normal(rows, 1)[0]
    (scale, se), (w, _), (wp, _), (bias, be), (bp, bpe) = (b.normal(1) for _ in range(5))
    (res, re_), (dro, droe), (dy, dye) = b.normal(rows, 1, dtype=rt), b.normal(rows, 1, dtype=rt), b.normal(rows, 1)
    kw = dict(res_dtype=rcode, kind="layer", post=True, pre=True, eps=1e-3)
    args = dict(w_post=wp, b_post=bp, scale=scale, res=res, w_pre=w, b_pre=bias)
    y, ro = b.out(rows, 1), b.out(rows, 1, dtype=rt)
    Q.SeqNormPlan(rows, 1, code, **kw).forward(x, y=y, res_out=ro, **args)
    assert np.array_equal(host(y), np.broadcast_to(be, (rows, 1)))
    O.check("res_out", host(ro), re_ + se * bpe, np.abs(re_) + np.abs(se * bpe), 4, rt == torch.bfloat16)
    g = {n: b.out(1, dtype=f32) for n in ("dw_post", "db_post", "dscale", "dw_pre", "db_pre")}
    dx, dr = b.out(rows, 1), b.out(rows, 1, dtype=rt)
    Q.SeqNormPlan(rows, 1, code, direction="bwd", **kw).backward(x, dx, dy=dy, dres_out=dro, dres=dr, **args, **g)
    assert not host(dx).any() and not host(g["dw_post"]).any() and not host(g["dw_pre"]).any()
    assert np.array_equal(host(dr), droe)
    for n, terms in (("db_post", droe * se), ("dscale", droe * bpe), ("db_pre", dye)):
        O.check(n, host(g[n]), terms.sum(0), np.abs(terms).sum(0), rows + 4, False)
    b.check_guards()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("lens,ragged", [([9, 3, 40, 0, 1, 700, 60], True), ([70] * 7, False), ([1] * 9, False), ([5] * 40, True)])
@pytest.mark.parametrize("D,pad", [(40, 0), (17, 1)])
def test_bad_values_stay_in_their_sequence(bf16, lens, ragged, D, pad):
    """Infinities and NaN in some sequences, in every input and state: the others' results have the bits that they have
    without them, and in the convolution and the scan so have the tokens before the first bad one."""
    import torch
    S, T, N, W = len(lens), sum(lens), 16, 4
    c = scan_case(T + D, bf16, lens, D, N, 1, pad=pad)
    b, dev, f32 = c["box"], c["dev"], torch.float32
    code, starts = CONV_BF16 if bf16 else CONV_F32, starts_of(lens) if ragged else None
    dev["dy"], dev["w"], dev["cbias"] = b.normal(T, D, pad=pad)[0], b.normal(D, W)[0], b.normal(D)[0]
    dev["h"], dev["dh"] = b.normal(S, D, N, dtype=f32)[0], b.normal(S, D, N, dtype=f32)[0]
    dev["cs"] = b.normal(S, W - 1, D)[0]
    bounds = O.bounds(lens)
    bad = [s for s in range(1, S, 2) if lens[s]]
    at = {s: bounds[s][0] + lens[s] // 2 for s in bad}           # the first bad token
    ok = np.ones(T, bool)
    before = np.ones(T, bool)
    for s in bad:
        ok[bounds[s][0]:bounds[s][1]] = False
        before[at[s]:bounds[s][1]] = False
    good_s = [s for s in range(S) if s not in bad]
    spoiled = {k: v.clone() for k, v in dev.items()}
    for i, s in enumerate(bad):
        for j, n in enumerate(("x", "dt", "B", "C", "z", "dy")):
            v = spoiled[n][at[s]:bounds[s][1]]
            v[:, (i + j) % 3::3] = (float("nan"), float("inf"), -float("inf"))[(i + j) % 3]
    states_spoiled = {k: spoiled[k].clone() for k in ("h", "dh", "cs")}
    for s in bad:
        for v in states_spoiled.values():
            v[s, ..., ::2] = float("nan")
    conv, conv_b = (Q.SeqConvPlan(S, T, D, W, code, direction=d, ragged=ragged) for d in ("fwd", "bwd"))
    scan, scan_b = (Q.SeqScanPlan(S, T, D, N, code, direction=d, ragged=ragged) for d in ("fwd", "bwd"))
    o = lambda *s, dtype=None: torch.zeros(*s, dtype=dtype or c["box"].t, device="cuda")      # noqa: E731

    def run(t):
        r = {n: o(T, D) for n in ("y", "dx", "sy", "sdx", "ddt", "dz")}
        r.update(dB=o(T, N), dC=o(T, N), cs=o(S, W - 1, D), h=o(S, D, N, dtype=f32), dh=o(S, D, N, dtype=f32))
        conv.forward(t["x"], t["w"], t["cbias"], r["y"], starts=starts, state_in=t["cs"], state_out=r["cs"])
        conv_b.backward(t["x"], t["w"], t["cbias"], t["dy"], r["dx"], o(D, W, dtype=f32), o(D, dtype=f32), starts=starts, state_in=t["cs"])
        arr, kw, saved = [t[n] for n in ("x", "dt", "A", "B", "C")], dict(D=t["D"], z=t["z"], dt_bias=t["dt_bias"], starts=starts), scan_b.allocate_saved()
        scan.forward(*arr, r["sy"], h_in=t["h"], h_out=r["h"], saved=saved, **kw)
        scan_b.backward(*arr, t["dy"], saved, r["sdx"], r["ddt"], o(D, N, dtype=f32), r["dB"], r["dC"], dz=r["dz"], dD=o(D, dtype=f32),
                        ddt_bias=o(D, dtype=f32), h_in=t["h"], dh_out=t["dh"], dh_in=r["dh"], **kw)
        return r

    clean, tokens, all_ = run(dev), run(spoiled), run({**spoiled, **states_spoiled})
    for n, v in clean.items():
        assert bool(torch.isfinite(v).all()), n
        rows = good_s if n in ("cs", "h", "dh") else torch.from_numpy(ok).cuda()
        assert torch.equal(tokens[n][rows], v[rows]) and torch.equal(all_[n][rows], v[rows]), n
        if n in ("y", "sy"):                      # what comes later does not reach back
            rows = torch.from_numpy(before).cuda()
            assert torch.equal(tokens[n][rows], v[rows]), n
    if T > 20:
        assert not bool(torch.isfinite(tokens["sy"]).all()) and not bool(torch.isfinite(tokens["y"]).all())


def test_bad_rows_of_a_norm_stay_bad_alone():
    import torch
    b = Box(8, True)
    for rows, D in ((9, 40), (7, 384), (9, 4096), (5, 9001)):
        x, g, dy = (b.normal(rows, D)[0] for _ in range(3))
        r, dr = (b.normal(rows, D, dtype=torch.float32)[0] for _ in range(2))
        w = b.normal(D)[0]
        ok = [i for i in range(rows) if i not in (1, 4)]
        for kind in ("rms", "layer"):
            f, q = (Q.SeqNormPlan(rows, D, CONV_BF16, d, kind=kind, post=True, gate="before") for d in ("fwd", "bwd"))

            def run():
                y, ro, dx, dg, dres = (torch.empty_like(t) for t in (x, r, x, g, r))
                f.forward(x, y=y, gate=g, w_post=w, res=r, res_out=ro, w_pre=w)
                q.backward(x, dx, dy=dy, gate=g, w_post=w, res=r, dres_out=dr, w_pre=w, dgate=dg, dres=dres)
                return y, ro, dx, dg, dres

            want = [t.clone() for t in run()]
            keep = [t.clone() for t in (x, g, r)]
            x[1, 3], g[4, ::2], r[4, 5] = float("nan"), float("inf"), -float("inf")
            for t, v in zip(run(), want):
                assert torch.equal(t[ok], v[ok])
            for t, v in zip((x, g, r), keep):
                t.copy_(v)
def test_decay_factors_have_no_bias():
    """Thousands of factors close to one, of sequences that are not cut.  A systematic 1.6e-8 below the true factor (what
    the special-function unit's 2^v has there) would leave every state 4096 times that, 6.6e-5, too small on average; the
    roundings of a state's own path, random, average out over 65536 states: half of 6.6e-5 separates the two."""
    import torch
    S, L, D, N = 512, 4096, 8, 16
    rng = np.random.default_rng(4)
    step = np.exp(rng.uniform(np.log(1e-3), np.log(1e-2), (S * L, D))).astype(np.float32)
    A = -rng.uniform(0.02, 0.1, (D, N)).astype(np.float32)
    h = rng.uniform(1, 2, (S, D, N)).astype(np.float32)
    put = lambda v: torch.from_numpy(v).cuda()      # noqa: E731
    p = Q.SeqScanPlan(S, S * L, D, N, CONV_F32, softplus=False)
    assert f"pieces={S} " in p.describe()
    z, bc = torch.zeros(S * L, D, device="cuda"), torch.zeros(S * L, N, device="cuda")
    y, left = torch.empty_like(z), torch.empty(S, D, N, device="cuda")
    p.forward(z, put(step), put(A), bc, bc, y, h_in=put(h), h_out=left)
    want = h.astype(np.float64) * np.exp(step.astype(np.float64).reshape(S, L, D).sum(1)[:, :, None] * A.astype(np.float64))
    off = host(left) / want - 1
    assert abs(off.mean()) < 0.5 * 1.6e-8 * L, off.mean()


@pytest.mark.parametrize("bf16", [False, True])
def test_steps_of_zero_keep_the_states(bf16):
    """delta = 0: a factor of exactly one and nothing added, over whole sequences and in steps."""
    import torch
    b = Box(1, bf16)
    S, L, D, N = 3, 50, 24, 16
    code, T = CONV_BF16 if bf16 else CONV_F32, 150
    x, B, C = b.normal(T, D)[0], b.normal(T, N)[0], b.normal(T, N)[0]
    A, h = b.put(-b.rng.uniform(0.01, 20, (D, N)), dtype=torch.float32)[0], b.normal(S, D, N, dtype=torch.float32)[0]
    dt, y, left = torch.zeros_like(x), torch.empty_like(x), torch.empty_like(h)
    Q.SeqScanPlan(S, T, D, N, code, softplus=False).forward(x, dt, A, B, C, y, h_in=h, h_out=left)
    assert torch.equal(left, h)
    Q.SeqScanPlan(S, S, D, N, code, direction="step", softplus=False).step(x[:S], dt[:S], A, B[:S], C[:S], h, left.zero_(), y[:S])
    assert torch.equal(left, h)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T", [300, 1300, 4100])
def test_growing_states_of_nothing_are_nothing(bf16, T):
    """A > 0: states grow by a third a token, by more than fp32 holds over a few pieces, but there is nothing to grow before
    the first input, nor a gradient behind the last one: zero, not infinity times zero."""
    import torch
    D, N, f32 = 24, 16, torch.float32
    b = Box(T, bf16)
    x, dy = b.rng.standard_normal((T, D)), b.rng.standard_normal((T, D))
    x[:-30], dy[30:] = 0, 0
    (x, xe), (dy, dye), (B, Be), (C, Ce) = b.put(x), b.put(dy), b.normal(T, N), b.normal(T, N)
    (dt, dte), (A, Ae) = b.put(np.ones((T, D))), b.put(b.rng.uniform(0.2, 0.4, (D, N)), dtype=f32)
    code = CONV_BF16 if bf16 else CONV_F32
    p, q = (Q.SeqScanPlan(1, T, D, N, code, direction=d, softplus=False) for d in ("fwd", "bwd"))
    assert int(p.describe().split("pieces=")[1].split()[0]) > 1
    y, saved, left = b.out(T, D), q.allocate_saved(), b.out(1, D, N, dtype=f32)
    p.forward(x, dt, A, B, C, y, h_out=left, saved=saved)
    g = {n: b.out(*s, dtype=f32 if n in ("dA", "dh_in") else None)
         for n, s in dict(dx=(T, D), ddt=(T, D), dA=(D, N), dB=(T, N), dC=(T, N), dh_in=(1, D, N)).items()}
    q.backward(x, dt, A, B, C, dy, saved, **g)
    ref, mag = O.scan(xe, dte, Ae, Be, Ce, 1, [T], np.zeros((1, D, N)), act=False, dy=dye)
    k = 4 * T + N + 100
    for n, v in dict(g, y=y, h=left).items():
        O.check(n, host(v), ref[n], mag[n], 2 * k + D + T, bf16 and v.dtype == torch.bfloat16)
    b.check_guards()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("starts", [[5, 3, 700, -4, 90, 12], [0, 1 << 30, -(1 << 30), 40, 40, 10], [400] * 6, [-1] * 6, [300, 250, 200, 150, 100, 50]])
@pytest.mark.parametrize("D,pad", [(40, 0), (17, 1)])
def test_bounds_outside_their_contract_write_nothing_elsewhere(bf16, starts, D, pad):
    """Other numbers, but the calls end and the outputs' surroundings are untouched.  (That no access leaves the
    tensors is shown on the host, from the lookups' own code.)"""
    import torch
    S, T, N, W, f32 = 5, 400, 16, 4, torch.float32
    b = Box(len(starts), bf16)
    code = CONV_BF16 if bf16 else CONV_F32
    n = lambda *s, **kw: b.normal(*s, **kw)[0]      # noqa: E731
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    slots = torch.tensor([2, -7, 1 << 30, 0, 1], dtype=torch.int32, device="cuda")
    x, dt, z, dy, B, C = n(T, D, pad=pad), n(T, D, pad=pad), n(T, D, pad=pad), n(T, D, pad=pad), n(T, N, pad=pad), n(T, N, pad=pad)
    w, bias, A, cs, h = n(D, W), n(D), -n(D, N, dtype=f32).abs(), n(3, W - 1, D), n(3, D, N, dtype=f32)
    o = lambda *s, dtype=None, p=pad: b.out(*s, dtype=dtype, pad=p)      # noqa: E731
    for direction in ("fwd", "bwd"):
        p = Q.SeqConvPlan(S, T, D, W, code, direction=direction, ragged=True)
        q = Q.SeqScanPlan(S, T, D, N, code, direction=direction, ragged=True)
        if direction == "fwd":
            p.forward(x, w, bias, o(T, D), starts=st, slots=slots, state_in=cs, state_out=o(3, W - 1, D, p=0))
            saved = q.allocate_saved().zero_()
            q.forward(x, dt, A, B, C, o(T, D), z=z, starts=st, slots=slots, h_in=h, h_out=o(3, D, N, dtype=f32, p=0), saved=saved)
        else:
            p.backward(x, w, bias, dy, o(T, D), o(D, W, dtype=f32, p=0), o(D, dtype=f32, p=0), starts=st, slots=slots, state_in=cs)
            q.backward(x, dt, A, B, C, dy, saved, o(T, D), o(T, D), o(D, N, dtype=f32, p=0), o(T, N), o(T, N), z=z, dz=o(T, D), starts=st, slots=slots,
                       h_in=h, dh_out=h, dh_in=o(3, D, N, dtype=f32, p=0))
        torch.cuda.synchronize()
    b.check_guards()
