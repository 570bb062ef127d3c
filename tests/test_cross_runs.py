"""Host checks of the number of runs that cross-attention's gradient cuts its sums
into: each kernel of a call finds it for itself, so it may not depend on how a
compiler treats floating point.  The choice is compiled from the kernels' own header."""
import ctypes
import os
import random
import shutil
import subprocess
from fractions import Fraction

import pytest

from exact_attention_68_gb300.build import CSRC, ROOT

SRC = os.path.join(ROOT, "tests", "cuda", "runs_check.cpp")


def _compile(to, *flags):
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    return subprocess.run([cxx, "-O2", "-std=c++17", "-I", CSRC, *flags, "-o", to, SRC], capture_output=True, text=True)


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    to = str(tmp_path_factory.mktemp("runs") / "libruns_check.so")
    r = _compile(to, "-fPIC", "-shared", "-fvisibility=hidden")
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(to)
    lib.runs_of.argtypes = [ctypes.c_int64] * 5 + [ctypes.c_int] * 3
    lib.most_runs.argtypes = [ctypes.c_int64] * 5 + [ctypes.c_int] * 2
    return lib


def test_the_choice_needs_no_floating_point(tmp_path):
    """With no registers for it, nothing of it is left to a compiler."""
    r = _compile(str(tmp_path / "runs_check.o"), "-c", "-mgeneral-regs-only")
    assert r.returncode == 0, r.stderr


def _width(D):
    return 64 if D <= 64 else 128 if D <= 128 else 256


def _times(D, rows, tiles, sms, most):
    """Expected times in us of 1 to `most` runs, exactly."""
    width = _width(D)
    step, ctas = (64, 2) if width == 256 else (128, 1)
    us = {64: Fraction(12, 10), 128: Fraction(19, 10), 256: Fraction(17, 10)}[width]
    steps = -(-rows // step)
    out = []
    for n in range(1, most + 1):
        t = -(-tiles * ctas * n // sms) * (-(-steps // n) + Fraction(3, 2)) * us
        out.append(t if n == 1 else t + 3 + Fraction(128 * D * 16, 5000000) * tiles * n)
    return out


def _check(shim, D, rows, tiles, sms):
    args = (1, tiles, 128, rows, D, _width(D), sms)
    t = _times(D, rows, tiles, sms, shim.most_runs(*args))
    n = shim.runs_of(*args, tiles)
    assert t[n - 1] < min(t) + Fraction(1, 1000), (D, rows, tiles, sms)  # whole nanoseconds
    return sorted(t)


def test_near_ties(shim):
    """Sizes where two numbers of runs cost the same to a part in 2^24, so that fp32 times with and without fused
    multiply-adds settled them differently."""
    for steps in (63, 83, 84, 103, 104, 124):
        first, second = _check(shim, 56, 128 * steps, 497, 152)[:2]
        assert second - first < first / 2 ** 24
        assert shim.runs_of(1, 497, 128, 128 * steps, 56, 64, 152, 497) == 2


def test_the_cheapest_number_of_runs(shim):
    rng = random.Random(1)
    for _ in range(4000):
        _check(shim, rng.randrange(8, 257, 8), rng.randrange(65, 40000), rng.randrange(1, 640), rng.choice([152, 148, 16]))


def test_bounds(shim):
    for rows, most in ((1, 1), (128, 1), (129, 2), (1000, 8), (1 << 30, 8)):
        assert shim.most_runs(1, 4, 128, rows, 64, 64, 152) == most
    assert shim.most_runs(1, 608, 128, 5000, 64, 64, 152) == 1 and shim.most_runs(1, 607, 128, 5000, 64, 64, 152) == 8
    assert shim.most_runs(1, 304, 128, 5000, 256, 256, 152) == 1
    # the longest sums do not overflow
    for tiles in (1, 500, 607):
        _check(shim, 128, (1 << 31) - 200, tiles, 152)
        _check(shim, 64, (1 << 31) - 200, tiles, 152)
    _check(shim, 256, (1 << 31) - 200, 303, 152)
