"""GPU tests of mla_window_bwd: what its rows of gradients do not depend on, and which rows of dkv
it writes."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

SENTINEL = 77.0


@pytest.fixture(scope="module")
def dsa():
    import sparse_attention_serving_gb300 as m
    return m


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _gradients(dsa, q, base, d_o, starts, window, first, dkv=None):
    B, T, H, _ = q.shape
    S = base.shape[1]
    rows, qs, kl = dsa.Rows(base), _i32(starts), _i32([v + T for v in starts])
    need = max(dsa.workspace_bytes(op, B, T, S, H, window + first)
               for op in (dsa.OP_MLA_WINDOW, dsa.OP_MLA_WINDOW_BWD))
    ws = dsa.new_workspace(need)
    o, lse = dsa.mla_window_fwd(q, rows, qs, kl, window, first, S, workspace=ws)
    dq, dkv = dsa.mla_window_bwd(q, rows, qs, kl, window, first, S, o, lse, d_o, dkv=dkv, workspace=ws)
    assert dsa.read_device_status(ws)[0] == dsa.DSA_OK
    return dq, dkv


@pytest.mark.parametrize("case", [(5, 60, 8, 77, 3), (3, 11, 96, 40, 4), (40, 1, 96, 200, 1), (2, 1500, 1, 130, 0)],
                         ids=str)
def test_gradients_alone_and_in_a_batch(dsa, case):
    """A sequence's dq has the same bits alone and in a batch (with more than 2048 rows, or less)."""
    B, T, H, window, first = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(60)
    S = 300 + T
    q, base, d_o = _normal(gen, B, T, H, 576), _normal(gen, B, S, 576), _normal(gen, B, T, H, 512)
    starts = [300 - 5 * b for b in range(B)]
    dq, _ = _gradients(dsa, q, base, d_o, starts, window, first)
    for b in {0, B // 2, B - 1}:
        one = slice(b, b + 1)
        alone, _ = _gradients(dsa, q[one].contiguous(), base[one].contiguous(), d_o[one].contiguous(),
                              starts[one], window, first)
        assert torch.equal(dq[b], alone[0]), b


def test_rows_of_a_sequence_without_queries(dsa):
    """Queries at or beyond kv_len see nothing and are flagged; the rows below kv_len get their zeros."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(61)
    B, T, H, S = 4, 3, 8, 600
    q, base, d_o = _normal(gen, B, T, H, 576), _normal(gen, B, S, 576), _normal(gen, B, T, H, 512)
    starts, lens = [597, 300, 520, 0], [600, 300, 257, 0]
    qs, kl = _i32(starts), _i32(lens)
    ws = dsa.new_workspace(dsa.workspace_bytes(dsa.OP_MLA_WINDOW_BWD, B, T, S, H, 90))
    dkv = torch.full((B, S, 576), SENTINEL, dtype=torch.bfloat16, device="cuda")
    o, lse = dsa.mla_window_fwd(q, dsa.Rows(base), qs, kl, 88, 2, S)
    dq, _ = dsa.mla_window_bwd(q, dsa.Rows(base), qs, kl, 88, 2, S, o, lse, d_o, dkv=dkv, workspace=ws)
    assert dsa.read_device_status(ws)[0] == dsa.DSA_ERR_BAD_INDEX
    assert (dq[1:] == 0).all()
    for b in range(B):
        assert (dkv[b, lens[b]:] == SENTINEL).all() and not (dkv[b, :lens[b]] == SENTINEL).any(), b
    for b in (1, 2):
        assert (dkv[b, :lens[b]] == 0).all(), b
    assert (dkv[0, 512:] != 0).any() and (dkv[0, 2:500] == 0).all()
