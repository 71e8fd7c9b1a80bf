"""GPU test of mla_tree_fwd, mla_window_fwd and mla_window_bwd: a workspace taken for the largest call
of a loop serves its smaller ones."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dsa():
    import sparse_attention_serving_gb300 as m
    return m


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_decode_batches_that_lose_a_request(dsa):
    """76 sequences may be done whole where 75 are cut."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(70)
    B, H, L = 76, 96, 1500
    ws = dsa.new_workspace(dsa.workspace_bytes(dsa.OP_MLA_TREE, B, 1, L + 1, H, 0))
    q, base = _normal(gen, B, 1, H, 576), _normal(gen, B, L + 1, 576)
    one = torch.ones((B, 1), dtype=torch.int64, device="cuda")
    for n in (76, 75, 40, 2, 1):
        args = q[:n].contiguous(), dsa.Rows(base[:n].contiguous()), one[:n].contiguous(), _i32([L] * n), L + 1
        o, lse = dsa.mla_tree_fwd(*args, workspace=ws)
        want, want_lse = dsa.mla_tree_fwd(*args)
        assert dsa.read_device_status(ws)[0] == dsa.DSA_OK
        assert torch.equal(o, want) and torch.equal(lse, want_lse), n


@pytest.mark.parametrize("case", [(2, 257, 8, 2500, 512, 4), (1, 700, 96, 700, 200, 0)], ids=str)
def test_chunks_that_get_shorter(dsa, case):
    B, T, H, S, window, first = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(71)
    ws = dsa.new_workspace(max(dsa.workspace_bytes(op, B, T, S, H, window + first)
                               for op in (dsa.OP_MLA_WINDOW, dsa.OP_MLA_WINDOW_BWD)))
    base = _normal(gen, B, S, 576)
    rows = dsa.Rows(base)
    for n in (T, T - 1, T // 2, 33, 1):
        q, d_o = _normal(gen, B, n, H, 576), _normal(gen, B, n, H, 512)
        args = q, rows, _i32([S - n] * B), _i32([S] * B), window, first, S
        o, lse = dsa.mla_window_fwd(*args, workspace=ws)
        want, want_lse = dsa.mla_window_fwd(*args)
        assert torch.equal(o, want) and torch.equal(lse, want_lse), n
        got = dsa.mla_window_bwd(*args, o, lse, d_o, workspace=ws)
        alone = dsa.mla_window_bwd(*args, o, lse, d_o)
        assert dsa.read_device_status(ws)[0] == dsa.DSA_OK
        assert torch.equal(got[0], alone[0]) and torch.equal(got[1], alone[1]), n
