"""Whether strided buffers of one call share a byte (CPU): column ranges of
one wider matrix do not.

tests/native/overlap_check.cpp drives rows_overlap of csrc/afx_internal.h
under AddressSanitizer and UndefinedBehaviorSanitizer, against sets of bytes.
"""
import os
import subprocess

from conftest import ROOT

CSRC = os.path.join(ROOT, "lossless_bf16_weight_afx_amd", "csrc")


def test_overlap(tmp_path):
    exe = tmp_path / "overlap_check"
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-pthread", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", "-I", CSRC,
                    os.path.join(ROOT, "tests", "native", "overlap_check.cpp"), "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "overlap ok" in r.stdout
