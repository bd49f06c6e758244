"""Which group norm calls join their entries in every block: cut out of the kernels' source and run on the host."""
from tests.test_delta_wait import build, cut


def test_blocks_join_few_entries(tmp_path):
    out = build(tmp_path, "gnorm_join_check", "gnorm_join.inc",
                [cut("seq_gnorm.cu", "constexpr int GT = ", ";"), "\n", cut("seq_gnorm.cu", "struct GnShape {", "\n};\n"), cut("seq_gnorm.cu", "GnShape gn_shape("),
                 cut("seq_gnorm.cu", "bool gn_self(")])
    assert out.returncode == 0 and " 0 wrong" in out.stdout, out.stdout + out.stderr
