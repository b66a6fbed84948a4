"""The row segments that the gated block's and the transposed product's
kernels decode (CPU).

tests/native/segment_check.cpp drives the functions of csrc/afx_index.h that
those kernels call, on streams of random code lengths, under
AddressSanitizer and UndefinedBehaviorSanitizer. A planted mistake in a copy
of the header must make it fail.
"""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "lossless_bf16_weight_afx_amd", "csrc")


def run(tmp_path, csrc):
    exe = tmp_path / "segment_check"
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", "-I", csrc,
                    os.path.join(ROOT, "tests", "native", "segment_check.cpp"), "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    return subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)


def test_segments(tmp_path):
    r = run(tmp_path, CSRC)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "segments ok" in r.stdout


@pytest.mark.parametrize("what,old,new", [
    ("the last segment's end taken from the chunk after the one it starts in",
     "return next & kSegLast ? stream_bits :", "return next & kSegLast ? base1 :"),
    ("the last segment's end taken for a group's", "const bool last = end >= left;", "const bool last = end > left;"),
    ("the end's chunk not told from the start's", "((in_chunk + end) / kChunk - ch) << 2", "0u"),
    ("word count unclamped", "return umin32(((end - ((uint32_t)wa << 5) + 31) >> 5) + 1, most);",
     "return ((end - ((uint32_t)wa << 5) + 31) >> 5) + 1;"),
    ("no word of look-ahead", "+ 31) >> 5) + 1, most);", "+ 31) >> 5), most);"),
])
def test_check_catches_a_planted_mistake(tmp_path, what, old, new):
    d = tmp_path / "pkg" / "csrc"
    shutil.copytree(CSRC, d)
    os.makedirs(tmp_path / "include")
    shutil.copy(os.path.join(ROOT, "include", "afx.h"), tmp_path / "include" / "afx.h")
    text = (d / "afx_index.h").read_text()
    assert text.count(old) == 1, what
    (d / "afx_index.h").write_text(text.replace(old, new))
    r = run(tmp_path, str(d))
    assert r.returncode != 0, f"{what}: the check did not notice\n{r.stdout}"
