"""The FP8 product's arithmetic on sizes (csrc/linear_plan.h), compiled for the host.
CPU only."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SHIM = """
#include "linear_plan.h"
extern "C" int row_bytes_left(int N, int n, int size, int most) {
  return dsa::lin::row_bytes_left(N, n, size, most);
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, so = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "sparse_attention_serving_gb300", "csrc"), str(src), "-o",
                    str(so)], check=True)
    return ctypes.CDLL(str(so))


@pytest.mark.parametrize("size", [2, 4])
@pytest.mark.parametrize("N", [1, 31, 32, 63, 64, 1001, (1 << 29) - 1, 1 << 29, (1 << 29) + 1,
                               (1 << 30) - 1])
def test_bytes_left_of_a_row(plan, N, size):
    """Against unbounded integers, at the first boxes of a row, its last ones, and behind
    it: with N near 2^30 an FP32 row is longer than 32 bits count."""
    per = 128 // size
    boxes = {0, 1, 2, N // per - 1, N // per, N // per + 1, N // per + 2}
    for n in sorted(per * b for b in boxes if b >= 0):
        want = min(128, (N - n) * size)
        got = plan.row_bytes_left(N, n, size, 128)
        assert got == want if want > 0 else got <= 0, (N, n, size, got, want)
