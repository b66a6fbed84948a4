"""The gated block's division of its slabs among workgroups (CPU).

tests/native/gated_split_check.cpp drives csrc/afx_gated_split.h, the
functions that the kernels and their launch code call, under
AddressSanitizer and UndefinedBehaviorSanitizer. A planted mistake in a copy
of the header must make it fail.
"""
import os
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "lossless_bf16_weight_afx_amd", "csrc")


def run(tmp_path, csrc):
    exe = tmp_path / "gated_split_check"
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", "-I", csrc,
                    os.path.join(ROOT, "tests", "native", "gated_split_check.cpp"), "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    return subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)


def test_gated_split(tmp_path):
    r = run(tmp_path, CSRC)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "gated split ok" in r.stdout


@pytest.mark.parametrize("what,old,new", [
    ("range found with a rounded-down quotient", "+ total - 1) / total - 1)", ") / total)"),
    ("one place too few", "s.most = (s.tile_slabs - 1) / least + 2;", "s.most = (s.tile_slabs - 1) / least + 1;"),
    ("ranges past the slabs", "total < resident ? total : resident", "resident"),
])
def test_check_catches_a_planted_mistake(tmp_path, what, old, new):
    d = tmp_path / "csrc"
    d.mkdir()
    text = open(os.path.join(CSRC, "afx_gated_split.h")).read()
    assert text.count(old) == 1, what
    (d / "afx_gated_split.h").write_text(text.replace(old, new))
    r = run(tmp_path, str(d))
    assert r.returncode != 0, f"{what}: the check did not notice\n{r.stdout}"
