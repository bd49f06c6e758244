"""Plans of the delta rule that cut the axis of long sequences: the rule that decides, the workspace, and the places that the kernels
look up, cut out of their sources and run on the host."""
import pytest

from convolution_forward_implicit_gb300 import delta as D
from convolution_forward_implicit_gb300 import seq as Q
from convolution_forward_implicit_gb300.binding import CONV_BF16, CONV_F32
from tests.test_delta_wait import D as DEVICE, build, cut


@pytest.fixture(scope="module")
def lib():
    from convolution_forward_implicit_gb300.build import build_library
    build_library()


def pieces(S, T, heads, Dk=128, Dv=128, code=CONV_BF16, ragged=True):
    p = D.SeqDeltaPlan(S, T, heads, heads, Dk, Dv, code, ragged=ragged)
    n = int(Q.seq_plan_describe(p.handle).split("piece_chunks=")[1])
    p.close()
    return n


@pytest.mark.parametrize("code", [CONV_BF16, CONV_F32])
def test_many_short_sequences_are_not_cut(lib, code):
    """Sequences whose lengths the plan does not know: one that holds most of the tokens may be cut, many short ones have nothing to cut."""
    for S in (40, 64, 256, 5000):
        for heads in (1, 8):
            assert pieces(S, 64 * S, heads, code=code) == 0 == pieces(S, 64 * S, heads, code=code, ragged=False)
    assert pieces(1, 4096, 8, code=code) == pieces(1, 4096, 8, code=code, ragged=False) > 0
    assert pieces(3, 6000, 2, code=code) > 0


def test_memory_goes_by_tokens_not_by_sequences(lib):
    """What pieces need is by their number, whatever the sequences'."""
    few, many = (D.SeqDeltaPlan(S, 16000, 1, 1, 64, 64, CONV_F32, ragged=True) for S in (20, 30))
    assert all(int(Q.seq_plan_describe(p.handle).split("piece_chunks=")[1]) > 0 for p in (few, many))
    chunk = 2 * 64 * 64 * 4 + 520 * 4                       # a chunk's matrices and row factors
    for p, S in ((few, 20), (many, 30)):
        run = int(Q.seq_plan_describe(p.handle).split("piece_chunks=")[1])
        marks = -(-16000 // (64 * run))
        assert p._ws_bytes <= (16000 // 64 + S) * chunk + marks * 3 * 64 * 64 * 4 + 6 * 256
        p.close()


def test_places_of_pieces(tmp_path):
    h = "__host__ __device__ inline long long "
    parts = [cut("seq_internal.h", DEVICE + "int seq_start("), cut("seq_internal.h", "struct CutPiece {", "\n};\n"), cut("seq_internal.h", h + "cut_slots("),
             cut("seq_internal.h", DEVICE + "int cut_base("), cut("seq_internal.h", DEVICE + "CutPiece cut_piece("), cut("seq_internal.h", h + "delta_marks("),
             cut("seq_internal.h", h + "delta_joined(", "}\n"), cut("seq_delta.cuh", "struct MarkPiece {", "\n};\n"), cut("seq_delta.cuh", DEVICE + "MarkPiece mark_piece("),
             cut("seq_delta.cuh", DEVICE + "int first_mark(", "}\n"), cut("seq_delta.cuh", "struct WalkPlace {", "\n};\n"), "template <int MODE>\n",
             cut("seq_delta.cuh", DEVICE + "WalkPlace walk_place(")]
    out = build(tmp_path, "delta_place_check", "delta_place.inc", parts)
    assert out.returncode == 0 and " 0 wrong" in out.stdout, out.stdout + out.stderr


@pytest.mark.parametrize("scale", [1e-50, -1e-60, 0.0, 2.0 ** -151])
def test_a_scale_too_small_for_fp32_is_refused(lib, scale):
    """Rounded to fp32 it is zero, which the C call takes for 1 / sqrt(Dk)."""
    with pytest.raises(ValueError):
        D.SeqDeltaPlan(1, 8, 1, 1, 16, 16, CONV_F32, scale=scale)
    D.SeqDeltaPlan(1, 8, 1, 1, 16, 16, CONV_F32, scale=2.0 ** -149).close()
