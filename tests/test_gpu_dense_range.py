"""GPU tests of mla_tree_fwd and mla_window_fwd where scores or values are far from one: what a
row's softmax is measured against, and P times V, have to stay in FP32's range."""
from __future__ import annotations

import math

import pytest
import torch

import dense_ref as ref

pytestmark = pytest.mark.gpu

DIM = 560                                   # a rotated dim: part of the scores, not of the values


@pytest.fixture(scope="module")
def dsa():
    import sparse_attention_serving_gb300 as m
    return m


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# B, T, H, rows before the queries, top row, tree
CASES = [
    (1, 1, 96, 400, 300, False),
    (1, 3, 40, 400, 300, False),
    (2, 600, 96, 400, 300, False),
    (1, 1, 96, 700, 300, True),
    (2, 5, 8, 5000, 2600, True),            # cut into pieces
    (16, 8, 96, 4096, 2600, True),
]


def _one_key(dsa, case, others, top, first_block, mixed):
    """Every query's scores are one exact product each, q . k = others for all keys and top for one, so
    far above that all weight is its (mixed: once or twice as much, from row to row): (o, lse, the key's
    values, its score)."""
    B, T, H, L, at, tree = case
    at = 70 if first_block else at
    gen = _gen(50)
    q = torch.zeros((B, T, H, 576), dtype=torch.bfloat16, device="cuda")
    q[..., DIM] = 2.0 ** 18
    if mixed:
        q[..., DIM] *= (1 + torch.rand((B, T, H), generator=gen, device="cuda")).to(torch.bfloat16)
    base = _normal(gen, B, L + T, 576)
    base[..., DIM] = others / 2 ** 18
    base[:, at, DIM] = top / 2 ** 18
    rows, kl = dsa.Rows(base), _i32([L] * B)
    if tree:
        masks = torch.ones((B, T), dtype=torch.int64, device="cuda") << torch.arange(T, device="cuda")
        op, call = dsa.OP_MLA_TREE, lambda ws: dsa.mla_tree_fwd(q, rows, masks, kl, L + T, workspace=ws)
    else:
        n = _i32([L + T] * B)
        op = dsa.OP_MLA_WINDOW
        call = lambda ws: dsa.mla_window_fwd(q, rows, kl, n, L + T, 0, L + T, workspace=ws)  # noqa: E731
    ws = dsa.new_workspace(dsa.workspace_bytes(op, B, T, L + T, H, 0 if tree else L + T))
    o, lse = call(ws)
    assert dsa.read_device_status(ws)[0] == dsa.DSA_OK
    z = q[..., DIM].double() * base[:, at, DIM].double()[:, None, None] * ref.SCALE
    return o, lse, base[:, at, :512].double()[:, None, None], z


SCORES = [
    # others, top, top in the first block, mixed; the exponent of the top's P in base 2 where its maximum
    # is a difference to the first block's, or (first block) an FP32 product
    (-5e10, 18200.0, False, False),          # -156
    (1e10, 5e10, False, False),              # -240
    (1e10, 3e10, False, False),              # -128
    (1e10, 6e10, False, False),              # 256
    (-3e9, 18200.0, False, False),           # 4
    (0.0, 5e11, True, False),                # -1216
    (0.0, 3e11, True, False),                # -256
    (0.0, 7e11, True, False),                # 1920
    (-5e10, 18200.0, False, True),
    (0.0, 5e11, True, True),
]


@pytest.mark.parametrize("scores", SCORES, ids=str)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_scores_far_from_zero(dsa, case, scores):
    """One key far above the others, all scores beyond 2^24: differences of scores are coarser than an
    exponent's range, yet the key's values are the answer.  P and the output are rounded to BF16 once
    each (off by HALF), the sum's reciprocal and FP32 steps by less than 2^-20; the log-sum-exp is the
    score, scaled and converted between bases in FP32 (four roundings)."""
    o, lse, v, z = _one_key(dsa, case, *scores)
    off = (2 * ref.HALF + ref.HALF ** 2 + 2.0 ** -20) * v.abs()
    ref.within(o, v.expand(o.shape), off.expand(o.shape), "o_lat")
    ref.within(lse, z, z.abs() * 2.0 ** -22, "lse")


@pytest.mark.parametrize("rise", [30.0, 55.0, -55.0])
@pytest.mark.parametrize("case", CASES + [(80, 1, 96, 500, 300, True), (77, 1, 128, 500, 300, False)], ids=str)
def test_large_values_behind_a_rise(dsa, case, rise):
    """Values of 2^100 behind scores that rise (from the first keys on, or above them) by less than what
    has a unit done again: P times V leaves FP32's range, the weighted mean does not."""
    B, T, H, L, at, tree = case
    gen = _gen(51)
    q = torch.zeros((B, T, H, 576), dtype=torch.bfloat16, device="cuda")
    q[..., DIM] = 1.0
    q[..., DIM + 1:] = _normal(gen, B, T, H, 576 - DIM - 1)
    base = _normal(gen, B, L + T, 576)
    base[..., :512] *= 2.0 ** 100
    base[..., DIM] = 0
    base[:, at:at + 3, DIM] = rise / ref.SCALE
    rows, kl = dsa.Rows(base), _i32([L] * B)
    masks = torch.ones((B, T), dtype=torch.int64, device="cuda") << torch.arange(T, device="cuda")
    t = torch.arange(L, L + T, device="cuda")[:, None]
    s = torch.arange(L + T, device="cuda")
    if tree:
        o, lse = dsa.mla_tree_fwd(q, rows, masks, kl, L + T)
        see = (s < L) | (s == t)
    else:
        o, lse = dsa.mla_window_fwd(q, rows, kl, _i32([L + T] * B), L + T, 0, L + T)
        see = s <= t
    for b in range(B):
        for i in range(0, T, 100):
            part = slice(i, min(i + 100, T))
            r_o, r_lse, o_off, lse_off = ref.forward(q[b, part], base[b], see[part])
            ref.within(o[b, part], r_o, o_off, "o_lat")
            ref.within(lse[b, part], r_lse, lse_off, "lse")


@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_a_row_that_all_see_makes_no_zeros(dsa, value):
    """A row of the prefix that holds an infinity or a NaN, and a rise: every token's outputs say so, as
    the formula's do; the next sequence's do not."""
    gen = _gen(52)
    B, T, H, L = 2, 4, 96, 700
    q, base = _normal(gen, B, T, H, 576), _normal(gen, B, L + T, 576)
    base[0, 300, 5] = value
    q[..., DIM] = 1.0
    base[:, 400, DIM] = 40.0 / ref.SCALE
    masks = torch.ones((B, T), dtype=torch.int64, device="cuda") << torch.arange(T, device="cuda")
    o, lse = dsa.mla_tree_fwd(q, dsa.Rows(base), masks, _i32([L] * B), L + T)
    z = torch.einsum("thr,nr->thn", q[0].double(), base[0].double())[..., 300]
    hit = z != -math.inf                                # there the weight is 0, and 0 * inf at dim 5
    assert not torch.isfinite(lse[0][hit] + o[0][hit].float().sum(-1)).any()
    if value == math.inf:
        assert torch.isfinite(lse[0][~hit]).all() and not torch.isfinite(o[0][~hit][:, 5]).any()
    see = torch.cat([torch.ones((T, L), dtype=torch.bool), torch.eye(T, dtype=torch.bool)], 1).cuda()
    r_o, r_lse, o_off, lse_off = ref.forward(q[1], base[1], see)
    ref.within(o[1], r_o, o_off, "o_lat")
    ref.within(lse[1], r_lse, lse_off, "lse")
