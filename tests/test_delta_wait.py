"""The bounded waits of the delta rule's tensor-core kernels, cut out of the kernels' sources and run on the host."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "convolution_forward_implicit_gb300", "csrc")


def cut(name, what, end="\n}\n"):
    text = open(os.path.join(SRC, name)).read()
    i = text.index(what)
    return text[i:text.index(end, i)] + end


def build(tmp_path, check, inc, parts):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("needs g++")
    (tmp_path / inc).write_text("".join(parts))
    exe = tmp_path / check
    subprocess.check_call([gxx, "-O1", "-std=c++17", "-pthread", "-I", str(tmp_path), os.path.join(ROOT, "tests", "native", check + ".cpp"), "-o", str(exe)])
    return subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)


D = "__device__ __forceinline__ "


def test_lanes_leave_a_wait_together(tmp_path):
    out = build(tmp_path, "delta_wait_check", "delta_wait.inc",
                [cut("seq_delta_tc.cuh", "constexpr long long WAIT_CYCLES", ";\n"), cut("seq_delta_tc.cuh", D + "bool wait_turn(")])
    assert out.returncode == 0 and " 0 wrong" in out.stdout, out.stdout + out.stderr


def test_a_walk_ends_with_nothing_on_its_way(tmp_path):
    out = build(tmp_path, "delta_settle_check", "delta_settle.inc",
                [cut("seq_delta_tc.cuh", "constexpr long long WAIT_CYCLES", ";\n"), cut("seq_delta_tc.cuh", D + "void settle("),
                 cut("seq_delta_tc.cu", "struct Turns {", "\n};\n")])
    assert out.returncode == 0 and " 0 wrong" in out.stdout, out.stdout + out.stderr
