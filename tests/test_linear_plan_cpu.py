"""The FP8 product's arithmetic on sizes (csrc/linear_plan.h), compiled for the host.
CPU only."""
import ctypes
import math
import os
import random
import subprocess

import pytest

from linear_kernels import KERNELS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SHIM = """
#include "linear_plan.h"
extern "C" int row_bytes_left(int N, int n, int size, int most) {
  return dsa::lin::row_bytes_left(N, n, size, most);
}
extern "C" long long pick(int M, int N, int K, int sms, int size, int* tokens, int* slices) {
  const dsa::lin::Pick at = dsa::lin::pick(M, N, (K + 127) / 128, sms, (long long)N * size);
  *tokens = at.nt;
  *slices = at.S;
  return at.nt == 0 ? 0 : dsa::lin::split_tiles(M, N, at.nt) * at.S;
}
extern "C" int take(int M, int N, int K, int sms, int size, int fits, int* tokens, int* slices) {
  int times = 0;    // the last one taken, and how many were tried
  dsa::lin::take_one_that_fits(M, N, (K + 127) / 128, sms, (long long)N * size,
                               [&](const dsa::lin::Pick& at) {
                                 ++times;
                                 *tokens = at.nt;
                                 *slices = at.S;
                                 return at.S <= 8 || fits != 0;
                               });
  return times;
}
extern "C" int offered(int tokens, int slices, int M, int N, int K) {
  return dsa::lin::offered(dsa::lin::Pick{tokens, slices}, M, N, (K + 127) / 128);
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
    lib = ctypes.CDLL(str(so))
    lib.pick.restype = ctypes.c_int64
    return lib


def _pick(plan, M, N, K, sms, size):
    t, s = ctypes.c_int(), ctypes.c_int()
    ctas = plan.pick(M, N, K, sms, size, ctypes.byref(t), ctypes.byref(s))
    return (t.value, s.value), ctas


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


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def test_every_choice_is_a_tested_kernel(plan):
    """KERNELS is what the GPU tests run one by one, whatever the choice takes."""
    rng = random.Random(1)
    seen = set()
    for _ in range(20000):
        M, N, K = _log(rng, 1, 20000), _log(rng, 1, 60000), 16 * _log(rng, 1, 1024)
        at, _ = _pick(plan, M, N, K, rng.choice([148, 152]), rng.choice([2, 4]))
        assert at in KERNELS and plan.offered(*at, M, N, K), (M, N, K, at)
        seen.add(at)
    assert len(seen) > 30 and (0, 1) in seen        # and the choice does use them


def test_offered_kernels(plan):
    many = 1 << 14
    got = {(t, s) for t in range(-1, 300) for s in range(-1, 40) if plan.offered(t, s, 1000, 1000, many)}
    assert got == set(KERNELS)
    for t, s in KERNELS:                            # at most one slice per 128 of K
        assert plan.offered(t, s, 1000, 1000, 128 * s)
        assert plan.offered(t, s, 1000, 1000, 128 * s - 112)
        assert s == 1 or not plan.offered(t, s, 1000, 1000, 128 * s - 128)
    assert not plan.offered(16, 16, 1 << 20, (1 << 20) - 1, many)   # 2^33 CTAs


def test_grids_of_the_largest_sizes(plan):
    """M, N, K < 2^30 and M * N < 2^40, as the entry point admits them."""
    top = (1 << 30) - 1
    for lm in range(31):
        for M in {min(top, 1 << lm), min(top, (1 << lm) + 1)}:
            limit = min(top, ((1 << 40) - 1) // M)
            for N in {limit, limit // 3 + 1, 1}:
                for K in (16, 128, 2048, 7168, 1 << 20, top - 15):
                    for sms in (8, 152):
                        at, ctas = _pick(plan, M, N, K, sms, 4)
                        assert at in KERNELS and ctas < 1 << 31, (M, N, K, at, ctas)


@pytest.mark.parametrize("M,N,K", [(64, 128, 7168), (1, 128, 7168), (16, 64, 12288), (1, 576, 7168),
                                   (64, 7168, 12288), (777, 1001, 1040)])
def test_clusters_above_eight_ctas_are_taken_only_where_they_fit(plan, M, N, K):
    t, s = ctypes.c_int(), ctypes.c_int()

    def take(fits):
        times = plan.take(M, N, K, 152, 4, fits, ctypes.byref(t), ctypes.byref(s))
        return times, (t.value, s.value)

    free, _ = _pick(plan, M, N, K, 152, 4)
    assert take(1) == (1, free)
    times, at = take(0)
    if free[1] <= 8:
        assert times == 1 and at == free
    else:
        assert times == 2 and at in KERNELS and at[1] <= 8 and plan.offered(*at, M, N, K)


def test_a_choice_with_large_clusters_is_among_those(plan):
    assert _pick(plan, 64, 128, 7168, 152, 4)[0][1] > 8
