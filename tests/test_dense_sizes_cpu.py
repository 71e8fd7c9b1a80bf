"""Workspace sizes of mla_tree_fwd, mla_window_fwd and mla_window_bwd that a caller takes for several
calls.  CPU only."""
import ctypes
import random

import pytest


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_attention_serving_gb300 as m
    return m


@pytest.mark.parametrize("H", [1, 3, 8, 40, 96, 128])
@pytest.mark.parametrize("op", ["OP_MLA_TREE", "OP_MLA_WINDOW", "OP_MLA_WINDOW_BWD"])
def test_workspace_of_the_largest_call_serves_the_smaller(dsa, op, H):
    """A size never falls as B, Tq, max_kv_len or the window grows."""
    op = getattr(dsa, op)
    most = 64 if op == dsa.OP_MLA_TREE else 16384

    def size(B, T, S, span):
        return dsa.workspace_bytes(op, B, T, S, H, span)

    # a step at a time along each
    for B, T, S, span in ((1, 1, 131072, 1028), (1, 8, 4096, 516), (3, 60, 700, 80), (16, 4, 9000, 300)):
        for k, steps in ((0, range(1, 170)), (1, range(1, min(most, 500))), (2, range(1, 3000, 7)),
                         (3, range(1, 3000, 11))):
            last, sizes = 0, [B, T, S, span]
            for v in steps:
                sizes[k] = v
                n = size(*sizes)
                assert n >= last, sizes
                last = n
    # and from any smaller call to any larger one
    rng = random.Random(H)

    def upto(hi):
        return round(hi ** rng.random())

    for _ in range(4000):
        large = [upto(256), upto(most), upto(131072), upto(8192)]
        small = [rng.choice((v, rng.randint(1, v), max(1, v - 1), upto(v))) for v in large]
        assert size(*small) <= size(*large), (small, large)


def test_workspace_stays_small_where_nothing_is_cut(dsa):
    """A few short sequences need no more than the status header."""
    for B, S in ((1, 512), (64, 512), (4, 100)):
        assert dsa.workspace_bytes(dsa.OP_MLA_TREE, B, 1, S, 96, 0) == 256


def test_positions_beyond_32_bits_are_refused(dsa):
    """A query's position, and the end of the last page, have to fit 32 bits (a pool of few pages may
    stand for any number of rows).  Refused calls do not get as far as a launch."""
    fake, ws = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 24)
    rows = dsa._Rows(1 << 20, 0, 1 << 20, 1 << 25, 64, 4)
    for S, T in ((2 ** 31 - 1, 1), (2 ** 31 - 65, 64), (2 ** 31 - 256, 1)):
        code = dsa.lib.mla_tree_fwd(fake, rows, fake, fake, None, 1, T, 96, S, 0.1, fake, fake, ws, 1 << 40, None)
        assert code == dsa.DSA_ERR_UNSUPPORTED, (S, T)
    for S, T in ((2 ** 31 - 1, 1), (2 ** 31 - 1, 4096), (2 ** 31 - 4096, 4096)):
        code = dsa.lib.mla_window_fwd(fake, rows, fake, fake, 1, T, 96, 64, 4, S, 0.1, fake, fake, ws, 1 << 40,
                                      None)
        assert code == dsa.DSA_ERR_UNSUPPORTED, (S, T)
