"""How programs use the sequence-mixing operators: streams that are not the current one, several host
threads, graphs."""
import pytest

from convolution_forward_implicit_gb300 import seq as Q
from convolution_forward_implicit_gb300.binding import CONV_F32

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
