"""Sizes of dsa_cache_append_rope beyond a launch's grid are refused.  CPU only: refused calls do not
get as far as a launch."""
import ctypes

import pytest

P = ctypes.c_void_p
FAKE, OTHER, WS = P(1 << 20), P(1 << 22), P(1 << 24)     # aligned, never dereferenced


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_attention_serving_gb300 as m
    return m


# CTAs of 128 items: 96 of a token's key and row, 4 of a head, 8 of an indexer head of 128
@pytest.mark.parametrize("sizes", [
    (4096, 8191, 1024, 1024, 128),      # 97 CTAs a token, 2^25 - 4096 tokens: 3.25e9
    (1, 22139007, 1024, 1024, 128),     # a token's CTAs beyond 2^31 - 1
    (31 * 2 ** 15, 32, 1024, 1024, 128),
    (2 ** 25 - 1, 1, 1024, 1024, 128),
    (2 ** 24, 2, 1, 1, 64),             # 2^25 tokens, whatever their size
], ids=str)
def test_tokens_beyond_the_grid_are_refused(dsa, sizes):
    B, T, H, HI, D = sizes
    rows = dsa._Rows(1 << 20, 64, 0, 0, 0, 0)
    code = dsa.lib.dsa_cache_append_rope(FAKE, FAKE, rows, rows, FAKE, FAKE, 10, None, None, FAKE, OTHER, H,
                                         FAKE, OTHER, HI, B, T, D, 1, 1, 1e-5, WS, 256, None)
    assert code == dsa.DSA_ERR_UNSUPPORTED
