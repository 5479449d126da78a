"""The addresses of the 8-bit product's stage loads, walked on the host."""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "error_feedback_quant_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_every_load_of_a_stage_lies_in_its_panel(tmp_path):
    exe = tmp_path / "stage_offsets_check"
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", CSRC, "-o", str(exe), os.path.join(HERE, "c", "stage_offsets_check.cpp")],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    loads, wrong, past = (int(v) for v in re.findall(r"=(\d+)", r.stdout))
    assert wrong == 0 and loads > 10 ** 6 and past > 0


def test_stage_loads_take_their_rows_from_the_checked_function():
    """The product's buffer loads have their row in the checked offset; the scalar offset is the stage's start alone."""
    text = open(os.path.join(CSRC, "echo_int8.hpp")).read()
    calls = re.findall(r"raw_ptr_buffer_load_lds\((.*?)\);", text, re.S)
    assert len(calls) == 1 and calls[0].endswith("lds, 16, off, k0, 0, 0"), calls
    uses = re.findall(r"(?<!void )stage_load16\((.*?)\);", text)
    assert uses and all(", off[i], k0, " in u for u in uses), uses
    assert re.findall(r"\boff\[i\] = (.*?)\(", text) == ["i < LM ? stage_offset"]
