"""The exponents of partial sums (no GPU): marks for zeros and for what is not
finite meet in no arithmetic that overflows.  The compiler refuses a constant
expression that does."""
import itertools
import os
import shutil
import subprocess

import pytest

CXX = shutil.which("g++") or shutil.which("clang++")
ZERO, BAD = -(1 << 31) // 4, (1 << 31) - 1
FINITE = (-163, -14, 0, 113)                   # of the smallest and the largest float32


def compiles(tmp_path, *lines):
    from zero_sharded_mixed_partition_amd import build as B
    src = tmp_path / "t.cpp"
    src.write_text("\n".join(['#include "part_exponent.h"', "using namespace zero_shard;", *lines]) + "\n")
    done = subprocess.run([CXX, "-std=c++17", "-fsyntax-only", f"-I{B.CSRC}", str(src)], capture_output=True, text=True)
    return done.returncode == 0, done.stderr


@pytest.mark.skipif(CXX is None, reason="no host compiler")
def test_shifts_do_not_overflow(tmp_path):
    checks = [f"static_assert(kAllZero == {ZERO} && kNotFinite == {BAD}, \"\");"]
    for e, top in itertools.product((ZERO, BAD) + FINITE, repeat=2):
        if e > top:
            continue                               # top is the largest of them
        want = 2 * (e - top) if e in FINITE and top in FINITE else 0
        checks.append(f"static_assert(({top} == kNotFinite ? 0 : part_shift({e}, {top})) == {want}, \"\");")
    ok, why = compiles(tmp_path, *checks)
    assert ok, why


@pytest.mark.skipif(CXX is None, reason="no host compiler")
def test_the_compiler_sees_an_overflow(tmp_path):
    """The difference formed before the marks are looked at is refused."""
    ok, why = compiles(tmp_path, "constexpr int top = kNotFinite, e = -14;", "constexpr int down = 2 * (e - top);")
    assert not ok and "overflow" in why
    assert os.path.exists(CXX)


def test_the_kernels_use_it():
    from zero_sharded_mixed_partition_amd import build as B
    text = open(os.path.join(B.CSRC, "orthogonalize_thin.hip")).read()
    assert "INT_MAX" not in text and "INT_MIN" not in text and text.count("part_shift(") == 2
    assert "bad = top == kNotFinite" in text and "bad ? 0 : part_shift(exponents[p], top)" in text
