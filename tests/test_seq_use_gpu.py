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
