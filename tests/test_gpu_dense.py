"""GPU tests of mla_tree_fwd, mla_window_fwd and mla_window_bwd against plain 64-bit forms
(dense_ref.py: the formulas and the bounds)."""
from __future__ import annotations

import math

import pytest
import torch

import dense_ref as ref

pytestmark = pytest.mark.gpu

SENTINEL = 77.0


@pytest.fixture(scope="module")
def dsa():
    import sparse_attention_serving_gb300 as m
    return m


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(gen, *shape, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _store(dsa, base, gen, is_paged):
    if not is_paged:
        return dsa.Rows(base), base, None
    pool, table = ref.paged(base, gen)
    return dsa.Rows(pool, table), pool, table


def _outputs(B, T, H):
    return (torch.full((B, T, H, 512), SENTINEL, dtype=torch.bfloat16, device="cuda"),
            torch.full((B, T, H), SENTINEL, device="cuda"))


def _ok(dsa, ws):
    assert dsa.read_device_status(ws)[0] == dsa.DSA_OK


# ---------------------------------------------------------------------------
# window
# ---------------------------------------------------------------------------

WINDOW_CASES = [
    # B, Tq, H, q_start, window, n_first, paged
    (1, 1, 96, [0], 1, 0, False),                  # the very first token
    (1, 1, 96, [0], 512, 4, True),
    (3, 1, 96, [5, 511, 700], 512, 4, True),       # decode, around the window's length
    (2, 1, 96, [3000, 64], 1000, 70, True),
    (5, 1, 8, [63, 64, 65, 127, 128], 64, 1, True),
    (1, 1, 1, [257], 100, 3, False),
    (2, 1, 128, [300, 40], 129, 0, True),
    (2, 5, 96, [60, 0], 64, 0, False),             # a page boundary inside the queries
    (1, 130, 8, [0], 1, 0, False),                 # every query its own row
    (2, 77, 8, [0, 200], 33, 5, False),
    (1, 200, 96, [0], 64, 0, False),
    (1, 67, 96, [450], 300, 16, True),
    (2, 33, 17, [100, 129], 128, 200, False),      # first tokens and window meet
    (1, 50, 128, [0], 1000, 0, True),              # window longer than the sequence
    (1, 9, 40, [500], 128, 4, True),
    (2, 20, 96, [30, 0], 0, 3, False),             # first tokens only
    (2, 3, 96, [70, 0], 0, 0, False),              # nothing at all
    (1, 300, 3, [77], 64, 64, False),
    (1, 4, 96, [4000], 2 ** 31 - 1, 2 ** 31 - 1, True),   # everything
    (70, 3, 5, [i * 7 for i in range(70)], 90, 2, True),
    # enough work for the largest tiles: some whole units, some cut ones
    (1, 260, 96, [100], 300, 5, True),
    (2, 401, 33, [0, 1000], 500, 65, False),
    (40, 3, 128, [20 * i for i in range(40)], 200, 1, True),
    (1, 3000, 1, [0], 200, 3, False),              # one head: a unit of 128 or more queries
]


def _window_case(dsa, case, seed, values=1.0):
    B, Tq, H, start, window, first, is_paged = case
    gen = _gen(seed)
    S = max(start) + Tq
    base = _normal(gen, B, S, 576, scale=values)
    base[:, :1] *= 2
    for b in range(B):
        base[b, start[b] + Tq:] = math.nan           # behind the sequence: anything
    rows, store, table = _store(dsa, base, gen, is_paged)
    q = _normal(gen, B, Tq, H, 576)
    return base, rows, q, _i32(start), _i32([v + Tq for v in start]), S


@pytest.mark.parametrize("case", WINDOW_CASES, ids=str)
def test_window_forward(dsa, case):
    B, Tq, H, start, window, first, _ = case
    base, rows, q, qs, kl, S = _window_case(dsa, case, 1)
    o, lse = _outputs(B, Tq, H)
    ws = dsa.new_workspace(dsa.workspace_bytes(dsa.OP_MLA_WINDOW, B, Tq, S, H, min(window + first, S)))
    dsa.mla_window_fwd(q, rows, qs, kl, window, first, S, o_lat=o, lse=lse, workspace=ws)
    _ok(dsa, ws)
    for b in range(B):
        n = start[b] + Tq
        see = ref.window_sees(torch.arange(start[b], n, device="cuda")[:, None],
                              torch.arange(n, device="cuda"), window, first)
        r_o, r_lse, o_off, lse_off = ref.forward(q[b], base[b, :n], see)
        ref.within(o[b], r_o, o_off, f"o_lat of sequence {b}")
        ref.within(lse[b], r_lse, lse_off, f"lse of sequence {b}")


def test_window_forward_makes_its_outputs(dsa):
    case = (2, 19, 8, [4, 0], 7, 1, False)
    base, rows, q, qs, kl, S = _window_case(dsa, case, 2)
    o, lse = dsa.mla_window_fwd(q, rows, qs, kl, 7, 1, S)
    o2, none = dsa.mla_window_fwd(q, rows, qs, kl, 7, 1, S, want_lse=False)
    assert none is None and torch.equal(o, o2) and lse.shape == (2, 19, 8)


@pytest.mark.parametrize("rise", [20.0, 600.0])
def test_window_forward_rising_scores(dsa, rise):
    """Scores that rise along the sequence by far more than an exponent holds: the softmax's
    reference has to move."""
    gen = _gen(3)
    B, Tq, H, S = 1, 130, 8, 900
    q = _normal(gen, B, Tq, H, 576)
    q[..., 0] = 16.0
    base = _normal(gen, B, S, 576)
    # dim 0 of row s: score rise * s / S, exactly representable steps
    base[0, :, 0] = (torch.arange(S, device="cuda") / S * rise / (16 * ref.SCALE)).to(torch.bfloat16)
    start = S - Tq
    o, lse = dsa.mla_window_fwd(q, dsa.Rows(base), _i32([start]), _i32([S]), 700, 4, S)
    see = ref.window_sees(torch.arange(start, S, device="cuda")[:, None],
                          torch.arange(S, device="cuda"), 700, 4)
    r_o, r_lse, o_off, lse_off = ref.forward(q[0], base[0], see)
    ref.within(o[0], r_o, o_off, "o_lat")
    ref.within(lse[0], r_lse, lse_off, "lse")


@pytest.mark.parametrize("case", [(2, 600, 96, 500, 4), (1, 20, 8, 300, 0), (3, 12, 8, 400, 2), (1, 1, 96, 900, 0)],
                         ids=str)
def test_window_units_done_twice(dsa, case):
    """Scores of some heads and of some queries that rise far beyond an exponent's range, for every
    number of rows that a CTA may hold."""
    B, Tq, H, window, first = case
    gen = _gen(40)
    S = 1000
    q, base = _normal(gen, B, Tq, H, 576), _normal(gen, B, S, 576)
    q[..., 0] = 0
    q[:, Tq // 3:, ::3, 0] = 16.0
    q[:, Tq // 2:, 1::5, 0] = -16.0
    base[..., 0] = (torch.arange(S, device="cuda") / S * 700 / (16 * ref.SCALE)).to(torch.bfloat16)
    start = S - Tq
    rows, qs, kl = dsa.Rows(base), _i32([start] * B), _i32([S] * B)
    ws = dsa.new_workspace(dsa.workspace_bytes(dsa.OP_MLA_WINDOW, B, Tq, S, H, window + first))
    o, lse = dsa.mla_window_fwd(q, rows, qs, kl, window, first, S, workspace=ws)
    again, _ = dsa.mla_window_fwd(q, rows, qs, kl, window, first, S, workspace=ws)
    _ok(dsa, ws)
    assert torch.equal(o, again)
    see = ref.window_sees(torch.arange(start, S, device="cuda")[:, None],
                          torch.arange(S, device="cuda"), window, first)
    for b in range(B):
        for at in range(0, Tq, 100):
            part = slice(at, min(at + 100, Tq))
            r_o, r_lse, o_off, lse_off = ref.forward(q[b, part], base[b], see[part])
            ref.within(o[b, part], r_o, o_off, "o_lat")
            ref.within(lse[b, part], r_lse, lse_off, "lse")


def test_window_more_units_than_are_done_twice(dsa):
    """Each pair of SMs holds more units than it can mark."""
    gen = _gen(41)
    H, window = 8, 200
    T = 76 * 1024 * 192 // H + 30000
    q = torch.zeros((1, T, H, 576), dtype=torch.bfloat16, device="cuda")
    base = torch.zeros((1, T, 576), dtype=torch.bfloat16, device="cuda")
    base[0] = _normal(gen, T, 576)
    q[0, :, :, :16] = _normal(gen, T, H, 16)
    # a page's last row may be far above the pages before: scores of 0, 111, 222 or 333
    q[..., 20] = 16.0
    page = torch.arange(T // 64, device="cuda")
    base[..., 20] = 0
    base[0, 63::64, 20] = (page % 4 * 96).to(torch.bfloat16)[:len(base[0, 63::64])]
    o, lse = dsa.mla_window_fwd(q, dsa.Rows(base), _i32([0]), _i32([T]), window, 0, T)
    for at in (0, 100000, T // 2, T - 40000, T - 64):
        t = torch.arange(at, at + 64, device="cuda")
        near = torch.arange(max(at - window, 0), at + 64, device="cuda")
        see = ref.window_sees(t[:, None], near, window, 0)
        r_o, r_lse, o_off, lse_off = ref.forward(q[0, t], base[0, near], see)
        ref.within(o[0, t], r_o, o_off, f"o_lat at {at}")
        ref.within(lse[0, t], r_lse, lse_off, f"lse at {at}")


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_window_row_reaches_only_who_sees_it(dsa, value):
    """A row that holds an infinity or a NaN: queries whose window has left it keep to the bounds
    (another path may compute them: its bits are its own)."""
    case = (1, 40, 8, [100], 16, 2, False)
    base, rows, q, qs, kl, S = _window_case(dsa, case, 4)
    at = 104
    base[0, at, 100] = value
    got, lse = dsa.mla_window_fwd(q, rows, qs, kl, 16, 2, S)
    t = torch.arange(100, 140, device="cuda")
    sees = (t >= at) & (t < at + 16)
    see = ref.window_sees(t[:, None], torch.arange(S, device="cuda"), 16, 2)[~sees]
    r_o, r_lse, o_off, lse_off = ref.forward(q[0, ~sees], base[0], see)
    ref.within(got[0, ~sees], r_o, o_off, "o_lat")
    ref.within(lse[0, ~sees], r_lse, lse_off, "lse")
    assert not torch.isfinite(lse[0, sees] + got[0, sees].float().sum(-1)).any()


def test_window_drops_pages_between(dsa):
    """Pages that no query sees may be gone from the table; one that is seen and is outside
    the pool is flagged, its rows not seen."""
    case = (1, 1, 96, [1000], 100, 4, True)
    base, rows, q, qs, kl, S = _window_case(dsa, case, 5)
    want, _ = dsa.mla_window_fwd(q, rows, qs, kl, 100, 4, S)
    ws = dsa.new_workspace(dsa.workspace_bytes(dsa.OP_MLA_WINDOW, 1, 1, S, 96, 104))
    rows.block_table[0, 1:14] = -7                      # rows 64..895
    got, _ = dsa.mla_window_fwd(q, rows, qs, kl, 100, 4, S, workspace=ws)
    _ok(dsa, ws)
    assert torch.equal(got, want)
    rows.block_table[0, 15] = 10 ** 6                   # rows 960..1000
    got, lse = dsa.mla_window_fwd(q, rows, qs, kl, 100, 4, S, workspace=ws)
    assert dsa.read_device_status(ws)[0] == dsa.DSA_ERR_BAD_INDEX
    see = ref.window_sees(torch.tensor([[1000]], device="cuda"), torch.arange(S, device="cuda"), 100, 4)
    see[:, 960:] = False
    r_o, r_lse, o_off, lse_off = ref.forward(q[0], base[0], see)
    ref.within(got[0], r_o, o_off, "o_lat")
    ref.within(lse[0], r_lse, lse_off, "lse")


def test_window_bad_lengths_are_flagged(dsa):
    """Queries beyond kv_len, a kv_len beyond max_kv_len, a negative start: nothing seen."""
    gen = _gen(6)
    q = _normal(gen, 4, 3, 8, 576)
    base = _normal(gen, 4, 40, 576)
    ws = dsa.new_workspace(dsa.workspace_bytes(dsa.OP_MLA_WINDOW, 4, 3, 40, 8, 9))
    qs, kl = _i32([10, 38, -1, 30]), _i32([13, 40, 5, 41])
    o, lse = dsa.mla_window_fwd(q, dsa.Rows(base), qs, kl, 8, 1, 40, workspace=ws)
    assert dsa.read_device_status(ws)[0] == dsa.DSA_ERR_BAD_INDEX
    assert torch.isfinite(lse[0]).all() and torch.isfinite(lse[1, :2]).all()
    for bad in (lse[1, 2:], lse[2], lse[3]):
        assert (bad == -math.inf).all()
    for bad in (o[1, 2:], o[2], o[3]):
        assert (bad == 0).all()


# ---------------------------------------------------------------------------
# tree
# ---------------------------------------------------------------------------

def _masks(seed, B, T, kind):
    pick = torch.Generator()
    pick.manual_seed(seed)
    out = []
    for _ in range(B):
        sees = []
        for j in range(T):
            if kind == "any":                          # any bits at all, later tokens' too
                v = sum(1 << k for k in range(64) if torch.randint(0, 2, (), generator=pick))
            else:
                parent = int(torch.randint(-1, j, (), generator=pick)) if j else -1
                v = (sees[parent] if parent >= 0 else 0) | 1 << j
            sees.append(v)
        out.append([0 if kind == "none" else v - (1 << 64) if v >> 63 else v for v in sees])
    return torch.tensor(out, dtype=torch.int64, device="cuda")


TREE_CASES = [
    # B, T, H, prefix, n_draft, masks, paged
    (1, 1, 96, [0], None, "tree", False),
    (1, 1, 96, [1], None, "tree", True),
    (4, 1, 96, [63, 64, 700, 2049], None, "tree", True),
    (2, 1, 8, [5000, 31], None, "tree", True),
    (3, 1, 128, [200, 0, 129], None, "tree", False),
    (2, 8, 96, [1000, 60], None, "tree", True),
    (3, 7, 8, [0, 64, 130], [7, 0, 3], "tree", False),
    (2, 33, 8, [100, 3], [33, 20], "tree", True),
    (2, 64, 3, [61, 500], None, "tree", True),
    (1, 64, 96, [90], None, "any", False),
    (2, 16, 40, [0, 10], None, "none", False),        # prefix or nothing
    (2, 5, 96, [0, 0], [5, 2], "any", True),
    (1, 3, 1, [300], None, "tree", False),
    (8, 16, 96, [1000, 0, 63, 700, 1500, 129, 64, 900], [16, 3, 16, 0, 1, 16, 9, 12], "tree", True),
    (3, 40, 96, [640, 2000, 1], None, "tree", False),
    (100, 2, 96, [5 * i for i in range(100)], None, "tree", True),
]


def _tree_case(dsa, case, seed):
    B, T, H, prefix, n_draft, kind, is_paged = case
    gen = _gen(seed)
    S = max(prefix) + T
    base = _normal(gen, B, S, 576)
    n = n_draft or [T] * B
    for b in range(B):
        base[b, prefix[b] + n[b]:] = math.nan
    rows, store, table = _store(dsa, base, gen, is_paged)
    return base, rows, _normal(gen, B, T, H, 576), _masks(seed, B, T, kind), n, S


def _tree_sees(masks, prefix, n, T):
    """[n, prefix + T]"""
    bits = torch.tensor([[v >> j & 1 for j in range(T)] for v in masks.tolist()],
                        dtype=torch.bool, device="cuda")
    bits[:, n:] = False
    return torch.cat([torch.ones((T, prefix), dtype=torch.bool, device="cuda"), bits], 1)[:n]


@pytest.mark.parametrize("case", TREE_CASES, ids=str)
def test_tree_forward(dsa, case):
    B, T, H, prefix, n_draft, _, _ = case
    base, rows, q, masks, n, S = _tree_case(dsa, case, 11)
    o, lse = _outputs(B, T, H)
    ws = dsa.new_workspace(dsa.workspace_bytes(dsa.OP_MLA_TREE, B, T, S, H, 0))
    dsa.mla_tree_fwd(q, rows, masks, _i32(prefix), S, n_draft=None if n_draft is None else _i32(n_draft),
                     o_lat=o, lse=lse, workspace=ws)
    _ok(dsa, ws)
    for b in range(B):
        see = _tree_sees(masks[b], prefix[b], n[b], T)[:, :prefix[b] + n[b]]
        r_o, r_lse, o_off, lse_off = ref.forward(q[b, :n[b]], base[b, :prefix[b] + n[b]], see)
        ref.within(o[b, :n[b]], r_o, o_off, f"o_lat of sequence {b}")
        ref.within(lse[b, :n[b]], r_lse, lse_off, f"lse of sequence {b}")
        assert (o[b, n[b]:] == SENTINEL).all() and (lse[b, n[b]:] == SENTINEL).all()


def test_tree_sibling_with_nan_is_not_seen(dsa):
    """Drafted token 1's row is a NaN: only the tokens that see it are touched."""
    case = (1, 4, 96, [70], None, "tree", False)
    base, rows, q, _, _, S = _tree_case(dsa, case, 12)
    masks = torch.tensor([[1, 2 | 1, 4 | 1, 8 | 2 | 1]], dtype=torch.int64, device="cuda")
    base[0, 71] = math.nan
    o, lse = dsa.mla_tree_fwd(q, rows, masks, _i32([70]), S)
    see = _tree_sees(masks[0], 70, 4, 4)[[0, 2]]
    r_o, r_lse, o_off, lse_off = ref.forward(q[0, [0, 2]], base[0], see)
    ref.within(o[0, [0, 2]], r_o, o_off, "o_lat")
    ref.within(lse[0, [0, 2]], r_lse, lse_off, "lse")
    assert torch.isnan(o[0, [1, 3]]).all()


def test_tree_bad_lengths_are_flagged(dsa):
    gen = _gen(13)
    q, base = _normal(gen, 4, 3, 8, 576), _normal(gen, 4, 40, 576)
    masks = _masks(13, 4, 3, "tree")
    ws = dsa.new_workspace(dsa.workspace_bytes(dsa.OP_MLA_TREE, 4, 3, 40, 8, 0))
    o, lse = dsa.mla_tree_fwd(q, dsa.Rows(base), masks, _i32([37, 38, -1, 30]), 40,
                              n_draft=_i32([3, 3, 1, 4]), workspace=ws)
    assert dsa.read_device_status(ws)[0] == dsa.DSA_ERR_BAD_INDEX
    assert torch.isfinite(lse[0]).all() and torch.isfinite(lse[3]).all()
    assert (lse[1] == -math.inf).all() and (lse[2, 0] == -math.inf).all() and (o[1] == 0).all()


def test_tree_counts_out_of_range(dsa):
    """n_draft below 0 and above T: taken as the nearer bound and flagged, also where a sequence
    then has no token at all."""
    gen = _gen(15)
    q, base = _normal(gen, 2, 3, 8, 576), _normal(gen, 2, 40, 576)
    masks = _masks(15, 2, 3, "tree")
    ws = dsa.new_workspace(dsa.workspace_bytes(dsa.OP_MLA_TREE, 2, 3, 40, 8, 0))
    want, _ = dsa.mla_tree_fwd(q, dsa.Rows(base), masks, _i32([10, 20]), 40, workspace=ws)
    _ok(dsa, ws)
    for counts, rows in (([3, -1], [3, 0]), ([9, 3], [3, 3]), ([-7, -7], [0, 0])):
        o, lse = _outputs(2, 3, 8)
        dsa.mla_tree_fwd(q, dsa.Rows(base), masks, _i32([10, 20]), 40, n_draft=_i32(counts), o_lat=o,
                         lse=lse, workspace=ws)
        assert dsa.read_device_status(ws)[0] == dsa.DSA_ERR_BAD_INDEX, counts
        for b in range(2):
            assert torch.equal(o[b, :rows[b]], want[b, :rows[b]])
            assert (o[b, rows[b]:] == SENTINEL).all() and (lse[b, rows[b]:] == SENTINEL).all()


@pytest.mark.parametrize("rise", [0.0, 300.0])
def test_tree_pieces_by_the_slow_path(dsa, rise):
    """A long prefix, cut into pieces: with scores that rise beyond an exponent's range, and with
    a sibling's NaN in the last piece."""
    gen = _gen(16)
    T, H, L = 3, 40, 5000
    q, base = _normal(gen, 1, T, H, 576), _normal(gen, 1, L + T, 576)
    q[..., 0] = 16.0
    if rise:
        base[0, :L, 0] = (torch.arange(L, device="cuda") / L * rise / (16 * ref.SCALE)).to(torch.bfloat16)
    base[0, L + 1] = math.nan
    masks = torch.tensor([[1, 3, 5]], dtype=torch.int64, device="cuda")
    o, lse = dsa.mla_tree_fwd(q, dsa.Rows(base), masks, _i32([L]), L + T)
    see = _tree_sees(masks[0], L, T, T)[[0, 2]]
    r_o, r_lse, o_off, lse_off = ref.forward(q[0, [0, 2]], base[0], see)
    ref.within(o[0, [0, 2]], r_o, o_off, "o_lat")
    ref.within(lse[0, [0, 2]], r_lse, lse_off, "lse")
    assert torch.isnan(o[0, 1]).all()


@pytest.mark.parametrize("case", [(1, 3, 40, 5000), (4, 8, 96, 6000), (1, 1, 96, 9000)], ids=str)
def test_tree_pieces_done_twice(dsa, case):
    """Pieces of a long prefix whose scores rise beyond an exponent's range within the piece."""
    B, T, H, L = case
    gen = _gen(42)
    q, base = _normal(gen, B, T, H, 576), _normal(gen, B, L + T, 576)
    q[:, :, ::2, 0] = 16.0
    wave = (torch.arange(L, device="cuda") % 500) / 500 * 600
    base[:, :L, 0] = (wave / (16 * ref.SCALE)).to(torch.bfloat16)
    masks = _masks(42, B, T, "tree")
    ws = dsa.new_workspace(dsa.workspace_bytes(dsa.OP_MLA_TREE, B, T, L + T, H, 0))
    o, lse = dsa.mla_tree_fwd(q, dsa.Rows(base), masks, _i32([L] * B), L + T, workspace=ws)
    _ok(dsa, ws)
    for b in range(B):
        r_o, r_lse, o_off, lse_off = ref.forward(q[b], base[b], _tree_sees(masks[b], L, T, T))
        ref.within(o[b], r_o, o_off, "o_lat")
        ref.within(lse[b], r_lse, lse_off, "lse")


@pytest.mark.parametrize("case", [(76, 1, 96, 16384), (76, 1, 96, 8192), (76, 1, 96, 64), (76, 1, 96, 0),
                                  (40, 8, 96, 4096), (90, 13, 8, 4096), (3, 1, 96, 65536)], ids=str)
def test_tree_odd_pages_that_all_share(dsa, case):
    """Odd numbers of pages and a cache that stays in L2: a block without a second page must not
    run ahead of the CTA that has none to copy."""
    gen = _gen(44)
    B, T, H, L = case
    pages = 400
    pool = _normal(gen, pages, 64, 576)
    P = L // 64 + 1
    table = (torch.arange(B * P, device="cuda") % pages).view(B, P).to(torch.int32).contiguous()
    rows, q, kl = dsa.Rows(pool, table), _normal(gen, B, T, H, 576), _i32([L] * B)
    masks = torch.full((B, T), (1 << T) - 1, dtype=torch.int64, device="cuda")
    ws = dsa.new_workspace(dsa.workspace_bytes(dsa.OP_MLA_TREE, B, T, L + T, H, 0))
    first, _ = dsa.mla_tree_fwd(q, rows, masks, kl, L + T, workspace=ws)
    for _ in range(40):
        o, lse = dsa.mla_tree_fwd(q, rows, masks, kl, L + T, workspace=ws)
        assert torch.equal(o, first)
    _ok(dsa, ws)
    see = torch.ones((T, L + T), dtype=torch.bool, device="cuda")
    for b in (0, B - 1):
        r_o, r_lse, o_off, lse_off = ref.forward(q[b], ref.logical(pool, table, b, L + T), see)
        ref.within(o[b], r_o, o_off, "o_lat")
        ref.within(lse[b], r_lse, lse_off, "lse")


def test_tree_long_row_by_row(dsa):
    """A sibling's NaN behind a prefix that takes seconds row by row: the waits last."""
    gen = _gen(43)
    B, T, H, pages = 152, 2, 96, 8192
    L = pages * 64 - 64
    pool = torch.empty((pages + B, 64, 576), dtype=torch.bfloat16, device="cuda")
    for at in range(0, pages + B, 1024):
        pool[at:at + 1024] = _normal(gen, min(1024, pages + B - at), 64, 576)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(B, 1)
    table[:, -1] = pages + torch.arange(B, device="cuda")
    pool[pages + 7, 1] = math.nan                     # drafted token 1 of sequence 7
    q = _normal(gen, B, T, H, 576)
    masks = torch.tensor([[1, 3]] * B, dtype=torch.int64, device="cuda")
    ws = dsa.new_workspace(dsa.workspace_bytes(dsa.OP_MLA_TREE, B, T, L + T, H, 0))
    rows = dsa.Rows(pool, table.contiguous())
    o, lse = dsa.mla_tree_fwd(q, rows, masks, _i32([L] * B), L + T, workspace=ws)
    _ok(dsa, ws)
    assert torch.isnan(o[7, 1]).all() and not torch.isnan(o[8:]).any()
    see = torch.ones((1, L + 1), dtype=torch.bool, device="cuda")
    for b, i in ((7, 0), (6, 0)):
        for h in range(0, H, 32):
            cache = ref.logical(pool, table, b, L + 1)
            r_o, r_lse, o_off, lse_off = ref.forward(q[b, i:i + 1, h:h + 32], cache, see)
            ref.within(o[b, i:i + 1, h:h + 32], r_o, o_off, "o_lat")
            ref.within(lse[b, i:i + 1, h:h + 32], r_lse, lse_off, "lse")


def test_tree_of_one_chain_is_the_window_without_end(dsa):
    """A chain of drafted tokens sees what causal queries see."""
    gen = _gen(14)
    q, base = _normal(gen, 1, 6, 96, 576), _normal(gen, 1, 206, 576)
    chain = torch.tensor([[(1 << i + 1) - 1 for i in range(6)]], dtype=torch.int64, device="cuda")
    o, lse = dsa.mla_tree_fwd(q, dsa.Rows(base), chain, _i32([200]), 206)
    w, w_lse = dsa.mla_window_fwd(q, dsa.Rows(base), _i32([200]), _i32([206]), 1000, 0, 206)
    see = ref.window_sees(torch.arange(200, 206, device="cuda")[:, None],
                          torch.arange(206, device="cuda"), 1000, 0)
    _, _, o_off, lse_off = ref.forward(q[0], base[0], see)
    ref.within(o[0], w[0].double(), 2 * o_off, "o_lat")
    ref.within(lse[0], w_lse[0].double(), 2 * lse_off, "lse")


# ---------------------------------------------------------------------------
# backward
# ---------------------------------------------------------------------------

BWD_CASES = [
    # B, Tq, H, q_start, window, n_first
    (1, 1, 96, [0], 1, 0),
    (1, 1, 1, [200], 65, 2),
    (2, 7, 8, [0, 130], 5, 1),
    (1, 130, 8, [0], 64, 0),
    (1, 70, 96, [0], 33, 3),
    (2, 40, 96, [100, 0], 70, 16),
    (1, 20, 128, [64], 20, 0),
    (1, 150, 17, [3], 100, 130),
    (1, 33, 40, [0], 1000, 0),
    (2, 5, 96, [70, 0], 0, 3),
    (2, 5, 3, [70, 0], 0, 0),
    (1, 300, 2, [0], 2 ** 31 - 1, 0),
    (1, 900, 3, [0], 10, 300),                     # first tokens in two key tiles
    (2, 700, 1, [500, 0], 260, 1),                 # one head: a tile of 128 queries
    (1, 200, 96, [0], 150, 4),                     # several tasks for each pair
]


def _bwd_case(dsa, case, seed):
    B, Tq, H, start, window, first = case
    base, rows, q, qs, kl, S = _window_case(dsa, (*case, False), seed)
    gen = _gen(seed + 1)
    d_o = _normal(gen, B, Tq, H, 512)
    o = torch.empty((B, Tq, H, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((B, Tq, H), device="cuda")
    sees = []
    for b in range(B):
        n = start[b] + Tq
        see = ref.window_sees(torch.arange(start[b], n, device="cuda")[:, None],
                              torch.arange(n, device="cuda"), window, first)
        r_o, r_lse, _, _ = ref.forward(q[b], base[b, :n], see)
        o[b], lse[b] = r_o.to(torch.bfloat16), r_lse.float()
        sees.append(see)
    return base, rows, q, qs, kl, S, o, lse, d_o, sees


@pytest.mark.parametrize("case", BWD_CASES, ids=str)
def test_window_backward(dsa, case):
    B, Tq, H, start, window, first = case
    base, rows, q, qs, kl, S, o, lse, d_o, sees = _bwd_case(dsa, case, 21)
    dq = torch.full((B, Tq, H, 576), SENTINEL, dtype=torch.bfloat16, device="cuda")
    dkv = torch.full((B, S, 576), SENTINEL, dtype=torch.bfloat16, device="cuda")
    ws = dsa.new_workspace(dsa.workspace_bytes(dsa.OP_MLA_WINDOW_BWD, B, Tq, S, H, min(window + first, S)))
    dsa.mla_window_bwd(q, rows, qs, kl, window, first, S, o, lse, d_o, dq=dq, dkv=dkv, workspace=ws)
    _ok(dsa, ws)
    for b in range(B):
        n = start[b] + Tq
        r_dq, r_dkv, dq_off, dkv_off = ref.backward(q[b], base[b, :n], sees[b], o[b], lse[b], d_o[b])
        ref.within(dq[b], r_dq, dq_off, f"dq of sequence {b}")
        ref.within(dkv[b, :n], r_dkv, dkv_off, f"dkv of sequence {b}")
        assert (dkv[b, n:] == SENTINEL).all()


def test_window_backward_against_differences(dsa):
    """Along random directions of q and of the rows: the kernel's gradients against central
    differences of the 64-bit forward."""
    case = (1, 40, 8, [10], 12, 2)
    base, rows, q, qs, kl, S, o, lse, d_o, sees = _bwd_case(dsa, case, 23)
    dq, dkv = dsa.mla_window_bwd(q, rows, qs, kl, 12, 2, S, o, lse, d_o)
    _, _, dq_off, dkv_off = ref.backward(q[0], base[0], sees[0], o[0], lse[0], d_o[0])
    gen = _gen(24)
    q64, kv64, g64 = q[0].double(), base[0].double(), d_o[0].double()

    def value(qq, kk):
        return float((ref.forward(qq, kk, sees[0])[0] * g64).sum())

    # what rounding o_lat to BF16 does to d_o . o_lat, and so to each dz
    p = torch.exp(torch.einsum("thr,nr->thn", q64, kv64) * ref.SCALE - lse[0].double()[..., None])
    p = torch.where(sees[0][:, None], p, 0.0)
    D_off = ref.HALF * torch.einsum("thv,thv->th", g64.abs(), o[0].double().abs())
    z_off = ref.SCALE * p * D_off[..., None]
    dq_off = dq_off + torch.einsum("thn,nr->thr", z_off, kv64.abs())
    dkv_off = dkv_off + torch.einsum("thn,thr->nr", z_off, q64.abs())
    for _ in range(4):
        u = torch.randn(q64.shape, generator=gen, device="cuda", dtype=torch.float64)
        w = torch.randn(kv64.shape, generator=gen, device="cuda", dtype=torch.float64)
        e = 1e-4
        for got, off, d, f in ((dq[0], dq_off, u, lambda x: value(q64 + x * u, kv64)),
                               (dkv[0], dkv_off, w, lambda x: value(q64, kv64 + x * w))):
            slope = (8 * (f(e) - f(-e)) - (f(2 * e) - f(-2 * e))) / (12 * e)
            along = float((got.double() * d).sum())
            assert abs(slope - along) <= float((off * d.abs()).sum()) + 1e-6 * abs(slope)


def test_window_backward_follows_its_forward(dsa):
    """Forward and backward as a training step runs them, with an accumulated loss."""
    gen = _gen(25)
    B, Tq, H, S, window, first = 2, 90, 96, 90, 40, 4
    base, q = _normal(gen, B, S, 576), _normal(gen, B, Tq, H, 576)
    d_o = _normal(gen, B, Tq, H, 512)
    rows, qs, kl = dsa.Rows(base), _i32([0, 0]), _i32([S, S])
    need = max(dsa.workspace_bytes(op, B, Tq, S, H, window + first)
               for op in (dsa.OP_MLA_WINDOW, dsa.OP_MLA_WINDOW_BWD))
    ws = dsa.new_workspace(need)
    o, lse = dsa.mla_window_fwd(q, rows, qs, kl, window, first, S, workspace=ws)
    dq, dkv = dsa.mla_window_bwd(q, rows, qs, kl, window, first, S, o, lse, d_o, workspace=ws)
    _ok(dsa, ws)
    t = torch.arange(S, device="cuda")
    see = ref.window_sees(t[:, None], t, window, first)
    for b in range(B):
        r_dq, r_dkv, dq_off, dkv_off = ref.backward(q[b], base[b], see, o[b], lse[b], d_o[b])
        ref.within(dq[b], r_dq, dq_off, "dq")
        ref.within(dkv[b], r_dkv, dkv_off, "dkv")


def test_window_backward_bad_sequence(dsa):
    """A sequence whose length is out of range: dq = 0, its dkv untouched, the others right."""
    gen = _gen(26)
    q, base, d_o = _normal(gen, 2, 3, 8, 576), _normal(gen, 2, 40, 576), _normal(gen, 2, 3, 8, 512)
    qs, kl = _i32([10, 30]), _i32([13, 41])
    ws = dsa.new_workspace(dsa.workspace_bytes(dsa.OP_MLA_WINDOW_BWD, 2, 3, 40, 8, 9))
    o = torch.zeros((2, 3, 8, 512), dtype=torch.bfloat16, device="cuda")
    dkv = torch.full((2, 40, 576), SENTINEL, dtype=torch.bfloat16, device="cuda")
    dq, _ = dsa.mla_window_bwd(q, dsa.Rows(base), qs, kl, 8, 1, 40, o, torch.zeros((2, 3, 8), device="cuda"),
                               d_o, dkv=dkv, workspace=ws)
    assert dsa.read_device_status(ws)[0] == dsa.DSA_ERR_BAD_INDEX
    assert (dq[1] == 0).all() and (dkv[1] == SENTINEL).all()
    assert (dkv[0, 13:] == SENTINEL).all() and (dkv[0, 3:13] != SENTINEL).any()


def test_window_backward_in_chunks(dsa):
    """More P and dZ than the workspace takes at a time: dkv's sums go on from chunk to chunk."""
    B, Tq, H, window, first = 8, 4224, 8, 4000, 70      # 4.6 GB of blocks, 4.3 at a time
    gen = _gen(27)
    base, q, d_o = _normal(gen, B, Tq, 576), _normal(gen, B, Tq, H, 576), _normal(gen, B, Tq, H, 512)
    rows, qs, kl = dsa.Rows(base), _i32([0] * B), _i32([Tq] * B)
    need = dsa.workspace_bytes(dsa.OP_MLA_WINDOW_BWD, B, Tq, Tq, H, window + first)
    ws = dsa.new_workspace(need)
    o, lse = dsa.mla_window_fwd(q, rows, qs, kl, window, first, Tq)
    dq, dkv = dsa.mla_window_bwd(q, rows, qs, kl, window, first, Tq, o, lse, d_o, workspace=ws)
    _ok(dsa, ws)
    t = torch.arange(Tq, device="cuda")
    see = ref.window_sees(t[:, None], t, window, first)
    for b in (0, B - 1):
        r_dkv = off = 0
        for h in range(H):                           # a head at a time: 64-bit scores of 4224 x 4224
            g, k, g_off, k_off = ref.backward(q[b, :, h:h + 1], base[b], see, o[b, :, h:h + 1],
                                              lse[b, :, h:h + 1], d_o[b, :, h:h + 1])
            ref.within(dq[b, :, h:h + 1], g, g_off, f"dq of {b}, head {h}")
            r_dkv, off = r_dkv + k, off + k_off
        # a head's bound counts Tq additions, a sum over all heads H times as many: their share
        # 2 Tq ADD of a bound that is at least (HALF + 2 Tq ADD) of the same magnitudes
        share = 2 * Tq * ref.ADD / (ref.HALF + 2 * Tq * ref.ADD)
        ref.within(dkv[b], r_dkv, off * (1 + (H - 1) * share), f"dkv of {b}")


def test_window_backward_last_chunk_in_part(dsa):
    """The last chunk holds some tiles of each sequence only: a pair of SMs passes over tasks."""
    B, Tq, H, window, first = 2, 5000, 96, 1000, 4       # 3750 tiles each, 3448 at a time
    gen = _gen(28)
    base, q, d_o = _normal(gen, B, Tq, 576), _normal(gen, B, Tq, H, 576), _normal(gen, B, Tq, H, 512)
    rows, qs, kl = dsa.Rows(base), _i32([0] * B), _i32([Tq] * B)
    ws = dsa.new_workspace(dsa.workspace_bytes(dsa.OP_MLA_WINDOW_BWD, B, Tq, Tq, H, window + first))
    o, lse = dsa.mla_window_fwd(q, rows, qs, kl, window, first, Tq)
    dq, dkv = dsa.mla_window_bwd(q, rows, qs, kl, window, first, Tq, o, lse, d_o, workspace=ws)
    for _ in range(3):
        dq2, dkv2 = dsa.mla_window_bwd(q, rows, qs, kl, window, first, Tq, o, lse, d_o, workspace=ws)
        assert torch.equal(dq, dq2) and torch.equal(dkv, dkv2)
    _ok(dsa, ws)
    near = torch.cat([torch.arange(first, device="cuda"), torch.arange(Tq - 1700, Tq, device="cuda")])
    for b in range(B):
        for at in range(Tq - 600, Tq, 100):
            t = torch.arange(at, at + 100, device="cuda")
            see = ref.window_sees(t[:, None], near, window, first)
            r_dq, _, dq_off, _ = ref.backward(q[b, t], base[b, near], see, o[b, t], lse[b, t], d_o[b, t])
            ref.within(dq[b, t], r_dq, dq_off, f"dq of {b} from {at}")


# ---------------------------------------------------------------------------
# both: equal bits, graphs, streams
# ---------------------------------------------------------------------------

def test_beside_other_streams(dsa):
    """Pairs of CTAs whose two do not start together, as SMs fall free one by one: training steps
    and decode steps on three streams, an FP8 product and large copies on two more."""
    gen = _gen(29)
    streams = [torch.cuda.Stream() for _ in range(5)]

    def step(B, Tq, H, start, window, first):
        S = start + Tq
        base, q, d_o = _normal(gen, B, S, 576), _normal(gen, B, Tq, H, 576), _normal(gen, B, Tq, H, 512)
        rows, qs, kl = dsa.Rows(base), _i32([start] * B), _i32([S] * B)
        ws = dsa.new_workspace(max(dsa.workspace_bytes(op, B, Tq, S, H, window + first)
                                   for op in (dsa.OP_MLA_WINDOW, dsa.OP_MLA_WINDOW_BWD)))
        o, lse = _outputs(B, Tq, H)
        dq, dkv = torch.zeros_like(q), torch.zeros_like(base)

        def run(s):
            dsa.mla_window_fwd(q, rows, qs, kl, window, first, S, o_lat=o, lse=lse, workspace=ws, stream=s)
            dsa.mla_window_bwd(q, rows, qs, kl, window, first, S, o, lse, d_o, dq=dq, dkv=dkv,
                               workspace=ws, stream=s)
        return run, (o, lse, dq, dkv), ws

    def decode(B, L, H):
        base, q = _normal(gen, B, L + 1, 576), _normal(gen, B, 1, H, 576)
        rows, kl, masks = dsa.Rows(base), _i32([L] * B), torch.ones((B, 1), dtype=torch.int64, device="cuda")
        ws = dsa.new_workspace(dsa.workspace_bytes(dsa.OP_MLA_TREE, B, 1, L + 1, H, 0))
        o, lse = _outputs(B, 1, H)
        return (lambda s: dsa.mla_tree_fwd(q, rows, masks, kl, L + 1, o_lat=o, lse=lse, workspace=ws, stream=s),
                (o, lse), ws)

    def product(M, N, K):
        codes, scale = dsa.dsa_quant_fp8(_normal(gen, M * K // 128, 128))
        w, w_scale = dsa.dsa_quant_fp8_weight(_normal(gen, N, K))
        codes, scale = codes.view(M, K), scale.view(M, K // 128)
        ws = dsa.new_workspace(dsa.workspace_bytes(dsa.OP_LINEAR_FP8, M, 1, K, N, 0))
        out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        return (lambda s: dsa.dsa_linear_fp8(codes, scale, w, w_scale, out=out, workspace=ws, stream=s),
                (out,), ws)

    jobs = [step(76, 5, 96, 700, 300, 70), step(76, 5, 8, 900, 64, 0), decode(16, 2000, 96),
            product(1024, 7168, 512)]
    want = []
    for run, outs, ws in jobs:
        run(None)
        _ok(dsa, ws)
        want.append([t.clone() for t in outs])
    big = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    copy = torch.empty_like(big)
    torch.cuda.synchronize()
    for i in range(600):
        for s, (run, _, _) in zip(streams, jobs):
            run(s)
        if i % 3 == 0:
            with torch.cuda.stream(streams[4]):
                copy.copy_(big)
    torch.cuda.synchronize()
    for (_, outs, ws), expected in zip(jobs, want):
        _ok(dsa, ws)
        assert all(torch.equal(a, b) for a, b in zip(outs, expected))


def test_equal_calls_give_equal_bits(dsa):
    case = (2, 100, 96, [0, 37], 50, 4, False)
    base, rows, q, qs, kl, S = _window_case(dsa, case, 31)
    first = dsa.mla_window_fwd(q, rows, qs, kl, 50, 4, S)
    for _ in range(3):
        again = dsa.mla_window_fwd(q, rows, qs, kl, 50, 4, S)
        assert all(torch.equal(x, y) for x, y in zip(first, again))
    d_o = _normal(_gen(32), 2, 100, 96, 512)
    base = torch.nan_to_num(base)
    rows = dsa.Rows(base)
    grads = dsa.mla_window_bwd(q, rows, qs, kl, 50, 4, S, *first, d_o)
    for _ in range(3):
        again = dsa.mla_window_bwd(q, rows, qs, kl, 50, 4, S, *first, d_o)
        assert all(torch.equal(x, y) for x, y in zip(grads, again))


def test_streams_and_graphs(dsa):
    """Two calls at once on streams of their own, and a captured call replayed on new inputs."""
    gen = _gen(33)
    S, H = 3000, 96
    base = _normal(gen, 2, S, 576)
    rows, kl = dsa.Rows(base), _i32([S - 4, 1000])
    masks = _masks(33, 2, 4, "tree")
    qs = [_normal(gen, 2, 4, H, 576) for _ in range(2)]
    need = dsa.workspace_bytes(dsa.OP_MLA_TREE, 2, 4, S, H, 0)
    work = [dsa.new_workspace(need) for _ in range(2)]
    want = [dsa.mla_tree_fwd(q, rows, masks, kl, S) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    torch.cuda.synchronize()
    for k in (0, 1):
        got[k] = dsa.mla_tree_fwd(qs[k], rows, masks, kl, S, workspace=work[k], stream=streams[k])
    torch.cuda.synchronize()
    for k in (0, 1):
        assert all(torch.equal(x, y) for x, y in zip(got[k], want[k]))
    q = qs[0].clone()
    o, lse = _outputs(2, 4, H)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.mla_tree_fwd(q, rows, masks, kl, S, o_lat=o, lse=lse, workspace=work[0])
    q.copy_(qs[1])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[1][0]) and torch.equal(lse, want[1][1])
    for ws in work:
        _ok(dsa, ws)


def test_window_step_in_a_graph(dsa):
    """Forward and backward captured together and replayed on other inputs, beside an eager call
    of the same operators with a workspace of its own."""
    gen = _gen(34)
    B, Tq, H, S, window, first = 2, 60, 96, 60, 30, 2
    qs, kl = _i32([0, 0]), _i32([S, S])
    need = max(dsa.workspace_bytes(op, B, Tq, S, H, window + first)
               for op in (dsa.OP_MLA_WINDOW, dsa.OP_MLA_WINDOW_BWD))
    sets = [[_normal(gen, B, S, 576), _normal(gen, B, Tq, H, 576), _normal(gen, B, Tq, H, 512)]
            for _ in range(2)]

    def step(base, q, d_o, ws, o=None, lse=None, dq=None, dkv=None):
        rows = dsa.Rows(base)
        o, lse = dsa.mla_window_fwd(q, rows, qs, kl, window, first, S, o_lat=o, lse=lse, workspace=ws)
        return (o, lse, *dsa.mla_window_bwd(q, rows, qs, kl, window, first, S, o, lse, d_o, dq=dq,
                                            dkv=dkv, workspace=ws))

    work = [dsa.new_workspace(need) for _ in range(2)]
    want = [step(*x, work[0]) for x in sets]
    held = [x.clone() for x in sets[0]]
    out = [torch.empty_like(x) for x in want[0]]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*held, work[0], *out)
    for k in (1, 0, 1):
        for x, y in zip(held, sets[k]):
            x.copy_(y)
        graph.replay()
        eager = step(*sets[1 - k], work[1])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want[k]))
        assert all(torch.equal(x, y) for x, y in zip(eager, want[1 - k]))
    for ws in work:
        _ok(dsa, ws)


def test_calls_in_a_row_share_a_workspace(dsa):
    """Different operators and sizes one after another on one stream, nothing between them: the
    launches overlap, their results and the bytes behind the workspace do not change."""
    gen = _gen(35)
    S, H = 1500, 96
    base = _normal(gen, 3, S, 576)
    rows = dsa.Rows(base)
    calls = []
    for B, T, kind in ((3, 1, "tree"), (1, 40, "window"), (2, 8, "tree"), (3, 300, "window"),
                       (1, 130, "bwd"), (2, 1, "window")):
        q = _normal(gen, B, T, H, 576)
        if kind == "tree":
            masks, kl = _masks(35, B, T, "tree"), _i32([S - T] * B)
            need = dsa.workspace_bytes(dsa.OP_MLA_TREE, B, T, S, H, 0)
            calls.append((need, lambda ws, q=q, m=masks, kl=kl: dsa.mla_tree_fwd(q, rows, m, kl, S, workspace=ws)))
        else:
            qs, kl = _i32([S - T] * B), _i32([S] * B)
            if kind == "window":
                need = dsa.workspace_bytes(dsa.OP_MLA_WINDOW, B, T, S, H, 204)
                calls.append((need, lambda ws, q=q, qs=qs, kl=kl: dsa.mla_window_fwd(
                    q, rows, qs, kl, 200, 4, S, workspace=ws)))
            else:
                o, lse = dsa.mla_window_fwd(q, rows, qs, kl, 200, 4, S)
                d_o = _normal(gen, B, T, H, 512)
                need = dsa.workspace_bytes(dsa.OP_MLA_WINDOW_BWD, B, T, S, H, 204)
                calls.append((need, lambda ws, q=q, qs=qs, kl=kl, o=o, lse=lse, d_o=d_o: dsa.mla_window_bwd(
                    q, rows, qs, kl, 200, 4, S, o, lse, d_o, workspace=ws)))
    want = []
    for need, call in calls:
        guard = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")
        ws = guard[:need]
        ws[:256] = 0
        want.append(call(ws))
        _ok(dsa, ws)
        assert (guard[need:] == 171).all()
    ws = dsa.new_workspace(max(need for need, _ in calls))
    for _ in range(3):
        got = [call(ws) for _, call in calls]
    torch.cuda.synchronize()
    _ok(dsa, ws)
    for x, y in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(x, y))


def test_rows_with_a_stride_of_their_own(dsa):
    """Sequences packed more tightly than their store's rows: kv as one run of rows."""
    gen = _gen(36)
    flat = _normal(gen, 1, 250, 576)
    q = _normal(gen, 2, 20, 8, 576)
    rows = dsa.Rows(flat, seq_stride=130)                 # sequences at rows 0 and 130, of 120
    qs, kl = _i32([100, 100]), _i32([120, 120])
    o, lse = dsa.mla_window_fwd(q, rows, qs, kl, 50, 2, 120)
    t = torch.arange(100, 120, device="cuda")
    see = ref.window_sees(t[:, None], torch.arange(120, device="cuda"), 50, 2)
    for b in range(2):
        r_o, r_lse, o_off, lse_off = ref.forward(q[b], flat[0, 130 * b:130 * b + 120], see)
        ref.within(o[b], r_o, o_off, "o_lat")
        ref.within(lse[b], r_lse, lse_off, "lse")


def test_beyond_32_bit_offsets(dsa):
    """Queries, outputs and a paged cache of more than 2^31 elements each."""
    gen = _gen(37)
    B, T, H, pages = 2, 21000, 96, 60000
    pool = torch.zeros((pages, 64, 576), dtype=torch.bfloat16, device="cuda")
    table = torch.arange(pages - 2 * 329, pages, device="cuda", dtype=torch.int32).view(2, 329).contiguous()
    pool[table.flatten().long()] = _normal(gen, 2 * 329, 64, 576)
    q = torch.empty((B, T, H, 576), dtype=torch.bfloat16, device="cuda")
    for b in range(B):
        q[b] = _normal(gen, T, H, 576)
    assert q.numel() > 2 ** 31 and pool.numel() > 2 ** 31
    rows = dsa.Rows(pool, table)
    o, lse = dsa.mla_window_fwd(q, rows, _i32([0, 0]), _i32([T, T]), 70, 2, T)
    cache = ref.logical(pool, table, 1, T)
    at = torch.arange(T - 40, T, device="cuda")
    near = torch.cat([torch.arange(2, device="cuda"), torch.arange(T - 200, T, device="cuda")])
    see = ref.window_sees(at[:, None], near, 70, 2)
    r_o, r_lse, o_off, lse_off = ref.forward(q[1, -40:], cache[near], see)
    ref.within(o[1, -40:], r_o, o_off, "o_lat")
    ref.within(lse[1, -40:], r_lse, lse_off, "lse")
    masks = torch.ones((B, 1), dtype=torch.int64, device="cuda")
    o, lse = dsa.mla_tree_fwd(q[:, -1:].contiguous(), rows, masks, _i32([T - 1, 2000]), T)
    see = torch.ones((1, T), dtype=torch.bool, device="cuda")
    r_o, r_lse, o_off, lse_off = ref.forward(q[0, -1:], ref.logical(pool, table, 0, T), see)
    ref.within(o[0], r_o, o_off, "o_lat")
    del o, lse
    d_o = torch.zeros((B, T, H, 512), dtype=torch.bfloat16, device="cuda")
    d_o[1, -40:] = _normal(gen, 40, H, 512)
    base = torch.stack([ref.logical(pool, table, b, T).to(torch.bfloat16) for b in range(B)])
    qs, kl = _i32([0, 0]), _i32([T, T])
    o, lse = dsa.mla_window_fwd(q, dsa.Rows(base), qs, kl, 70, 2, T)
    dq, dkv = dsa.mla_window_bwd(q, dsa.Rows(base), qs, kl, 70, 2, T, o, lse, d_o)
    see = ref.window_sees(at[:, None], near, 70, 2)
    r_dq, r_dkv, dq_off, dkv_off = ref.backward(q[1, -40:], cache[near], see, o[1, -40:], lse[1, -40:],
                                                d_o[1, -40:])
    ref.within(dq[1, -40:], r_dq, dq_off, "dq")
    ref.within(dkv[1][near], r_dkv, dkv_off, "dkv")


# ---------------------------------------------------------------------------
# refusals of the binding
# ---------------------------------------------------------------------------

def _refusals(call, good, wrong):
    call(**good)
    for name, values in wrong.items():
        for v in values:
            with pytest.raises((TypeError, ValueError, RuntimeError)) as e:
                call(**{**good, name: v})
            assert "CUDA error" not in str(e.value), (name, v, e.value)


def _other(t):
    """Of another type, one short, strided, and on the CPU."""
    wide = torch.empty((*t.shape[:-1], 2 * t.shape[-1]), dtype=t.dtype, device="cuda")
    return [None, t.to(torch.float16), t[..., :-1].contiguous(), wide[..., ::2], t.cpu()]


def test_binding_refusals(dsa):
    gen = _gen(41)
    B, T, H, S = 2, 3, 8, 70
    base, q = _normal(gen, B, S, 576), _normal(gen, B, T, H, 576)
    o, lse = _outputs(B, T, H)
    kl, rows = _i32([67, 67]), dsa.Rows(base)
    ws = dsa.new_workspace(1 << 26)
    stores = [None, base, dsa.Rows(base[:1].contiguous()), dsa.Rows(base[..., :512].contiguous()),
              dsa.Rows(torch.zeros((B, S, 576), dtype=torch.uint8, device="cuda")),
              dsa.Rows(*ref.paged(base[:1].contiguous(), gen))]
    sizes = [0, -1, 1 << 31, 2.5, S + 1]
    masks = _masks(41, B, T, "tree")
    common = dict(q_lat=_other(q)[1:], kv=stores, kv_len=_other(kl), max_kv_len=sizes, o_lat=_other(o)[1:],
                  lse=_other(lse)[1:], scale=[0.0, -1.0, math.nan],
                  workspace=[torch.zeros(64, dtype=torch.uint8, device="cuda"), ws.cpu(), ws.float()])
    _refusals(dsa.mla_tree_fwd,
              dict(q_lat=q, kv=rows, tree=masks, kv_len=kl, max_kv_len=S, o_lat=o, lse=lse, workspace=ws),
              dict(common, tree=_other(masks), n_draft=_other(kl)[1:]))
    window = dict(q_lat=q, kv=rows, q_start=kl - 3, kv_len=kl, window=9, n_first=1, max_kv_len=S, o_lat=o,
                  lse=lse, workspace=ws)
    spans = dict(q_start=_other(kl), window=[-1, 1 << 31, 1.5, None], n_first=[-1, 1 << 31, "1"])
    _refusals(dsa.mla_window_fwd, window, dict(common, **spans))
    d_o, dkv = _normal(gen, B, T, H, 512), torch.zeros_like(base)
    _refusals(dsa.mla_window_bwd, dict(window, d_o=d_o, dkv=dkv, dq=torch.empty_like(q)),
              dict(common, **spans, d_o=_other(d_o), dkv=_other(dkv)[1:], dq=_other(q)[1:],
                   kv=stores + [dsa.Rows(*ref.paged(base, gen))]))
    torch.cuda.synchronize()


def test_append_binding_refusals(dsa):
    gen = _gen(42)
    B, T, S = 2, 3, 40
    k_pre, kv_new = torch.randn((B, T, 128), device="cuda"), _normal(gen, B, T, 576)
    k, v = torch.zeros((B, S, 128), dtype=torch.bfloat16, device="cuda"), _normal(gen, B, S, 576)
    q_pe, q_lat, q_idx = _normal(gen, B, T, 8, 64), _normal(gen, B, T, 8, 576), _normal(gen, B, T, 4, 128)
    table, qs, pos = torch.zeros((50, 64), device="cuda"), _i32([1, 2]), _i32([[0, 1, 2]] * 2)
    good = dict(k_pre=k_pre, kv_new=kv_new, k_cache=dsa.Rows(k), kv_cache=dsa.Rows(v), q_start=qs,
                rope=table, pos=pos, n_new=qs, q_pe=q_pe, q_lat=q_lat, q_idx=q_idx,
                q_idx_out=torch.empty_like(q_idx))
    _refusals(dsa.dsa_cache_append_rope, good,
              dict(k_pre=_other(k_pre), kv_new=_other(kv_new), k_cache=[None, k, dsa.Rows(v)],
                   kv_cache=[None, v, dsa.Rows(k), dsa.Rows(v[:1].contiguous())], q_start=_other(qs),
                   rope=_other(table), pos=_other(pos)[1:], n_new=_other(qs)[1:], q_pe=_other(q_pe),
                   q_lat=_other(q_lat), q_idx=_other(q_idx), q_idx_out=_other(q_idx)[1:],
                   kv_style=[-1, 3], key_style=[7], eps=[-1.0, math.nan, math.inf]))
    torch.cuda.synchronize()
