"""The search for a row's sequence, walked on the host for every number of
sequences that a call may have."""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "error_feedback_quant_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_a_wave_looks_at_places_that_are_there_and_finds_the_last(tmp_path):
    exe = tmp_path / "wave_search_check"
    subprocess.run(["g++", "-O2", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC, "-o", str(exe),
                    os.path.join(HERE, "c", "wave_search_check.cpp")], check=True)

    def walk(*args):
        r = subprocess.run([str(exe), *args], capture_output=True, text=True, timeout=300)
        return r.returncode, [int(v) for v in re.findall(r"=(\d+)", r.stdout)], r.stderr
    rc, (looked, outside, wrong), err = walk()
    assert rc == 0 and outside == 0 and wrong == 0 and looked > 10 ** 4, err
    # signed numbers, in which the last places of the largest searches wrap
    rc, (looked, outside, wrong), err = walk("signed")
    assert rc != 0 and outside > 0 and wrong > 0, err


def test_the_kernels_search_by_the_checked_form():
    text = open(os.path.join(CSRC, "echo_cache.hpp")).read()
    body = text[text.index("int last_at_most("):text.index("// whether row t is")]
    assert re.findall(r"s\.(\w+)\(", body) == ["turn", "place", "narrow"] and "WaveSearch s((uint32_t)n)" in body
