"""How programs use the sequence-mixing operators: streams that are not the current one, several host
threads, graphs."""
import pytest

from convolution_forward_implicit_gb300 import seq as Q
from convolution_forward_implicit_gb300.binding import CONV_BF16, CONV_F32

pytestmark = pytest.mark.gpu


def scan_inputs(T, D, N, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")      # noqa: E731
    return n(T, D), n(T, D) - 1, -torch.rand(D, N, generator=g, device="cuda") - 0.1, n(T, N), n(T, N)


# ---------------------------------------------------------------------------------- streams
T_, D_, N_ = 4100, 136, 16           # cut into pieces: the states between them pass through the workspace


def scan_reference():
    import torch
    a = scan_inputs(T_, D_, N_)
    want = torch.empty(T_, D_, device="cuda")
    p = Q.SeqScanPlan(1, T_, D_, N_, CONV_F32)
    assert Q.seq_workspace_bytes(p.handle) > 1 << 20
    p.forward(*a, want)
    torch.cuda.synchronize()
    return a, want


def test_first_call_on_a_stream_beside_pending_work():
    """Memory freed on the current stream while its kernels still run is not the workspace of a call elsewhere."""
    import torch
    a, want = scan_reference()
    p = Q.SeqScanPlan(1, T_, D_, N_, CONV_F32)
    y = torch.empty(T_, D_, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    junk = torch.empty(Q.seq_workspace_bytes(p.handle), dtype=torch.uint8, device="cuda")
    at = junk.data_ptr()
    torch.cuda._sleep(2_000_000)
    for i in range(200):
        junk.fill_(i % 256)
    del junk
    for _ in range(20):
        p.forward(*a, y, stream=side.cuda_stream)
    assert p.workspace.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_plan_dropped_while_its_stream_runs():
    """The workspace of a plan that is gone stays out of the current stream's hands until its own stream is done."""
    import torch
    a, want = scan_reference()
    p = Q.SeqScanPlan(1, T_, D_, N_, CONV_F32).allocate()
    y = torch.empty(T_, D_, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
    p.forward(*a, y, stream=side.cuda_stream)
    at, n = p.workspace.data_ptr(), Q.seq_workspace_bytes(p.handle)
    p.close()
    del p
    for _ in range(4):
        t = torch.empty(n, dtype=torch.uint8, device="cuda")
        assert t.data_ptr() != at
        t.fill_(255)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_one_plan_on_two_streams():
    import torch
    a, want = scan_reference()
    p = Q.SeqScanPlan(1, T_, D_, N_, CONV_F32)
    sides = [torch.cuda.Stream() for _ in range(2)]
    ys = [torch.empty(T_, D_, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, y in zip(sides, ys):
            with torch.cuda.stream(s):
                p.forward(*a, y)
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in ys)


# ---------------------------------------------------------------------------- host threads
def test_norm_gradients_from_two_host_threads():
    """Plans of other flags share a kernel and want other amounts of shared memory of it; calls with workspaces
    of their own may come from any threads."""
    import sys
    import threading
    import torch
    rows, D = 3, 4096
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s, dtype=torch.bfloat16: torch.randn(*s, generator=g, device="cuda").to(dtype)      # noqa: E731
    x, gate, dy = n(rows, D), n(rows, D), n(rows, D)
    res, dro = n(rows, D, dtype=torch.float32), n(rows, D, dtype=torch.float32)
    e = torch.empty_like

    def large():
        p = Q.SeqNormPlan(rows, D, CONV_BF16, "bwd", post=True, pre=True, gate=Q.SEQ_GATE_BEFORE)
        dx, dg, dr = e(x), e(gate), e(res)
        return lambda: p.backward(x, dx, dy=dy, gate=gate, res=res, dres_out=dro, dgate=dg, dres=dr), (dx, dg, dr)

    def small():
        p = Q.SeqNormPlan(rows, D, CONV_BF16, "bwd", post=True, pre=False, residual=False, gate=Q.SEQ_GATE_BEFORE)
        dx, dg = e(x), e(gate)
        return lambda: p.backward(x, dx, dy=dy, gate=gate, dgate=dg), (dx, dg)

    made = [large(), small()]
    want = []
    for call, out in made:
        call()
        torch.cuda.synchronize()
        want.append([t.clone() for t in out])
    errors = []

    def work(call):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30000):
                    call()
                torch.cuda.current_stream().synchronize()
        except Exception as exc:      # noqa: BLE001
            errors.append(exc)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(call,)) for call, _ in made]
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)          # (so that a thread is ready to go on when the other one enters the library)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    assert not errors, errors
    for (_, out), w in zip(made, want):
        assert all(torch.equal(a, b) for a, b in zip(out, w))


# ---------------------------------------------------------------------- arguments at any place
def shifted(t, by=1):
    """The same values, `by` elements behind an aligned address."""
    import torch
    flat = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)[by:].view(t.shape)
    flat.copy_(t)
    return flat


def strided(t, ld, by):
    import torch
    rows = torch.empty(t.shape[0], ld, dtype=t.dtype, device=t.device)[:, by:by + t.shape[1]]
    rows.copy_(t)
    return rows


@pytest.mark.parametrize("bf16", [False, True])
def test_arguments_read_by_elements_lie_anywhere(bf16):
    """Bounds, slots, parameters read one by one, the scan's B and C, and parameter gradients beside aligned rows: the
    same bits wherever they lie."""
    import torch
    code, T, D, N, W, lens = (CONV_BF16 if bf16 else CONV_F32), 300, 256, 16, 4, [100, 0, 200]
    g = torch.Generator(device="cuda").manual_seed(1)
    td, f32 = torch.bfloat16 if bf16 else torch.float32, torch.float32
    n = lambda *s, dtype=td: torch.randn(*s, generator=g, device="cuda").to(dtype)      # noqa: E731
    o = lambda *s, dtype=td: torch.zeros(*s, dtype=dtype, device="cuda")      # noqa: E731
    starts = torch.tensor([0, 100, 100, 300], dtype=torch.int32, device="cuda")
    slots = torch.tensor([1, 2, 0], dtype=torch.int32, device="cuda")

    def same(call, plain, moved):
        want = [t.clone() for t in call(plain)]
        got = call({**plain, **moved})
        assert all(torch.equal(a, b) for a, b in zip(got, want))

    # convolution
    p, q = (Q.SeqConvPlan(3, T, D, W, code, d, ragged=True) for d in ("fwd", "bwd"))
    a = dict(x=n(T, D), w=n(D, W), bias=n(D), starts=starts, slots=slots, state_in=n(3, W - 1, D))
    more = dict(dy=n(T, D), dw=o(D, W, dtype=f32), dbias=o(D, dtype=f32))
    moved = {k: shifted(a[k]) for k in ("w", "bias", "starts", "slots")}

    def conv(t):
        y, s = o(T, D), o(3, W - 1, D)
        p.forward(t["x"], t["w"], t["bias"], y, starts=t["starts"], slots=t["slots"], state_in=t["state_in"], state_out=s)
        return y, s

    def conv_back(t):
        dx = o(T, D)
        q.backward(t["x"], t["w"], t["bias"], t["dy"], dx, t["dw"], t["dbias"], starts=t["starts"], slots=t["slots"], state_in=t["state_in"])
        return dx, t["dw"], t["dbias"]

    same(conv, a, moved)
    same(conv_back, {**a, **more}, {**moved, "dw": shifted(more["dw"]), "dbias": shifted(more["dbias"])})

    # scan
    p, q = (Q.SeqScanPlan(3, T, D, N, code, d, ragged=True) for d in ("fwd", "bwd"))
    a = dict(x=n(T, D), dt=n(T, D) - 1, A=-n(D, N, dtype=f32).abs(), B=n(T, N), C=n(T, N), D=n(D, dtype=f32), z=n(T, D), dt_bias=n(D, dtype=f32),
             starts=starts, slots=slots, h_in=n(3, D, N, dtype=f32))
    moved = {k: shifted(a[k]) for k in ("D", "dt_bias", "starts", "slots", "h_in")}
    moved.update(B=strided(a["B"], 79 + 2 * N, 79), C=strided(a["C"], 79 + 2 * N, 79 + N))      # a projection of odd width
    saved = q.allocate_saved()

    def scan(t):
        y, h = o(T, D), o(3, D, N, dtype=f32)
        p.forward(t["x"], t["dt"], t["A"], t["B"], t["C"], y, D=t["D"], z=t["z"], dt_bias=t["dt_bias"], starts=t["starts"], slots=t["slots"],
                  h_in=t["h_in"], h_out=h, saved=saved)
        return y, h

    def scan_back(t):
        out = dict(dx=o(T, D), ddt=o(T, D), dz=o(T, D), **{k: t.get(k, v) for k, v in
                   dict(dA=o(D, N, dtype=f32), dB=o(T, N), dC=o(T, N), dD=o(D, dtype=f32), ddt_bias=o(D, dtype=f32)).items()})
        q.backward(t["x"], t["dt"], t["A"], t["B"], t["C"], t["dy"], saved, D=t["D"], z=t["z"], dt_bias=t["dt_bias"], starts=t["starts"],
                   slots=t["slots"], h_in=t["h_in"], **out)
        return tuple(out.values())

    same(scan, a, moved)
    b = {**a, "dy": n(T, D)}
    moved.update(dA=shifted(o(D, N, dtype=f32)), dD=shifted(o(D, dtype=f32)), ddt_bias=shifted(o(D, dtype=f32)), dB=strided(o(T, N), N + 3, 3),
                 dC=strided(o(T, N), N + 3, 1))
    same(scan_back, b, moved)

    # norm
    q = Q.SeqNormPlan(T, D, code, "bwd", post=True)
    a = dict(x=n(T, D), dy=n(T, D), res=n(T, D, dtype=f32), w_post=n(D), w_pre=n(D), dw_post=o(D, dtype=f32), dw_pre=o(D, dtype=f32))

    def norm_back(t):
        dx, dr = o(T, D), o(T, D, dtype=f32)
        q.backward(t["x"], dx, dy=t["dy"], res=t["res"], w_post=t["w_post"], w_pre=t["w_pre"], dres=dr, dw_post=t["dw_post"], dw_pre=t["dw_pre"])
        return dx, dr, t["dw_post"], t["dw_pre"]

    same(norm_back, a, {k: shifted(a[k]) for k in ("dw_post", "dw_pre")})


# ----------------------------------------------------------------------------------- graphs
def test_a_training_step_in_a_graph():
    """Forward and backward calls of all three operators captured once and replayed on other inputs."""
    import torch
    S, L, D, N, W = 2, 600, 72, 16, 4
    T, bf, f32 = S * L, torch.bfloat16, torch.float32
    g = torch.Generator(device="cuda").manual_seed(5)
    n = lambda *s, dtype=bf: torch.randn(*s, generator=g, device="cuda").to(dtype)      # noqa: E731
    e = lambda *s, dtype=bf: torch.empty(*s, dtype=dtype, device="cuda")      # noqa: E731
    t = dict(x=n(T, D), dt=n(T, D) - 1, B=n(T, N), C=n(T, N), z=n(T, D), dy=n(T, D), res=n(T, D, dtype=f32))
    w, bias, nw, A, Dv = n(D, W), n(D), n(D), -n(D, N, dtype=f32).abs() - 0.1, n(D, dtype=f32)
    o = dict(cx=e(T, D), y=e(T, D), normed=e(T, D), r=e(T, D, dtype=f32), dx=e(T, D), ddt=e(T, D), dz=e(T, D), dB=e(T, N), dC=e(T, N), dA=e(D, N, dtype=f32),
             dD=e(D, dtype=f32), dcx=e(T, D), dw=e(D, W, dtype=f32), dbias=e(D, dtype=f32), dr=e(T, D, dtype=f32), dnw=e(D, dtype=f32), dn=e(T, D))
    conv, conv_b = (Q.SeqConvPlan(S, T, D, W, CONV_BF16, d).allocate() for d in ("fwd", "bwd"))
    scan, scan_b = (Q.SeqScanPlan(S, T, D, N, CONV_BF16, d).allocate() for d in ("fwd", "bwd"))
    norm, norm_b = (Q.SeqNormPlan(T, D, CONV_BF16, d).allocate() for d in ("fwd", "bwd"))
    saved = scan_b.allocate_saved()

    def step():
        conv.forward(t["x"], w, bias, o["cx"])
        a = (o["cx"], t["dt"], A, t["B"], t["C"])
        scan.forward(*a, o["y"], D=Dv, z=t["z"], saved=saved)
        norm.forward(o["y"], y=o["normed"], res=t["res"], res_out=o["r"], w_pre=nw)
        norm_b.backward(o["y"], o["dn"], dy=t["dy"], res=t["res"], w_pre=nw, dres=o["dr"], dw_pre=o["dnw"])
        scan_b.backward(*a, o["dn"], saved, o["dx"], o["ddt"], o["dA"], o["dB"], o["dC"], D=Dv, z=t["z"], dz=o["dz"], dD=o["dD"])
        conv_b.backward(t["x"], w, bias, o["dx"], o["dcx"], o["dw"], o["dbias"])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for v in t.values():
            v.copy_(torch.randn(v.shape, generator=g, device="cuda"))
        step()
        torch.cuda.synchronize()
        want = {k: v.clone() for k, v in o.items()}
        for v in o.values():
            v.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(v, want[k]) for k, v in o.items())


def test_a_call_captured_before_any_other():
    """Without a workspace at hand the captured call allocates one of the graph's own memory."""
    import torch
    a, want = scan_reference()
    p = Q.SeqScanPlan(1, T_, D_, N_, CONV_F32)
    y = torch.empty(T_, D_, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.forward(*a, y)
    for _ in range(2):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    p.forward(*a, y.zero_())                 # and an ordinary call behind it
    torch.cuda.synchronize()
    assert torch.equal(y, want)
