"""Calls of the delta rule without tokens: states and their gradients are handed on, and what follows in the stream finds them."""
import pytest

from convolution_forward_implicit_gb300 import delta as D
from tests.test_delta_gpu import CODE
from tests.test_seq_gpu import Box

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("S,H,K", [(3, 2, 64), (2500, 8, 128)])
def test_no_tokens(bf16, ragged, S, H, K):
    import torch
    b = Box(S, bf16)
    none = lambda w, dtype=b.t: torch.empty(0, w, dtype=dtype, device="cuda")      # noqa: E731
    f32 = torch.float32
    ins = [none(H * K), none(H * K), none(H * K), none(H, f32), none(H, f32)]
    starts = torch.zeros(S + 1, dtype=torch.int32, device="cuda") if ragged else None
    fwd, bwd = (D.SeqDeltaPlan(S, 0, H, H, K, K, CODE[bf16], d, ragged=ragged).allocate() for d in ("fwd", "bwd"))
    saved = bwd.allocate_saved()
    gen = torch.Generator("cuda").manual_seed(S)
    h = torch.randn(S, H, K, K, generator=gen, device="cuda")
    for _ in range(3):
        left, got = torch.full_like(h, 7.0), torch.empty_like(h)
        fwd.forward(*ins, none(H * K), starts=starts, h_in=h, h_out=left, saved=saved)
        got.copy_(left)
        assert torch.equal(got, h)
        left.fill_(7.0)
        bwd.backward(*ins, none(H * K), saved, *(torch.empty_like(t) for t in ins), starts=starts, dh_out=h, dh_in=left)
        got.copy_(left)
        assert torch.equal(got, h)
