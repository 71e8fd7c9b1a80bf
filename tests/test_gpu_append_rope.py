"""GPU tests of dsa_cache_append_rope against a plain 64-bit form.

A rotated value is a product, a second product and their sum in FP32 (each off by at most
2^-24 of its size, or less where they contract), so it lies within 3 * 2^-24 (|a c| + |b s|) of the
exact one before its one rounding to BF16; the key adds its LayerNorm's error (parity.py) through
both terms."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import dense_ref as ref
from parity import check_bf16_of, layernorm_delta

pytestmark = pytest.mark.gpu

EPS = 1e-5
SENTINEL = 77.0


@pytest.fixture(scope="module")
def dsa():
    import sparse_attention_serving_gb300 as m
    return m


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _table(n):
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(32) / 32)
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda()


def _turn(x, off, table, style):
    """x [..., 64] (64 bits) known to within off -> rotated values and their bounds."""
    if style == 0:
        return x, off
    c, s = table[..., :32], table[..., 32:]
    a, b = (x[..., :32], x[..., 32:]) if style == 1 else (x[..., 0::2], x[..., 1::2])
    da, db = (off[..., :32], off[..., 32:]) if style == 1 else (off[..., 0::2], off[..., 1::2])
    lo, hi = a * c - b * s, b * c + a * s
    d_lo = da * np.abs(c) + db * np.abs(s) + 3 * 2.0 ** -24 * (np.abs(a * c) + np.abs(b * s))
    d_hi = db * np.abs(c) + da * np.abs(s) + 3 * 2.0 ** -24 * (np.abs(b * c) + np.abs(a * s))
    if style == 1:
        return np.concatenate([lo, hi], -1), np.concatenate([d_lo, d_hi], -1)
    return (np.stack([lo, hi], -1).reshape(x.shape), np.stack([d_lo, d_hi], -1).reshape(x.shape))


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _np(t):
    return t.double().cpu().numpy()


CASES = [
    # B, Tq, D, heads, index heads, q_start, n_new, kv style, key style, paged, own positions, q_idx in place
    (1, 1, 128, 96, 64, [0], None, 2, 1, True, False, False),
    (1, 1, 64, 8, 4, [70], None, 1, 2, False, False, True),
    (5, 1, 128, 96, 64, [0, 63, 64, 300, 2048], None, 1, 1, True, False, False),
    (3, 8, 128, 8, 64, [60, 0, 121], [8, 0, 5], 2, 2, True, True, False),
    (2, 5, 64, 3, 4, [10, 0], [1, 5], 2, 2, False, True, False),
    (2, 33, 128, 1, 1, [100, 0], None, 0, 1, False, False, True),
    (2, 33, 128, 5, 7, [100, 0], None, 1, 0, True, True, True),
    (1, 700, 128, 17, 64, [321], None, 2, 1, True, False, False),
    (1, 9, 64, 128, 0, [0], None, 1, 1, False, False, False),      # no indexer queries
    (2, 4, 128, 0, 64, [9, 77], None, 1, 1, False, False, False),  # no absorbed queries
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_append_rope(dsa, case):
    B, T, D, H, HI, start, n_new, kv_style, key_style, is_paged, own_pos, in_place = case
    gen = _gen(hash(case[:5]) % 1000)
    S = max(start) + T
    table = _table(S + 5)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)

    k_base = torch.full((B, S, D), SENTINEL, dtype=torch.bfloat16, device="cuda")
    v_base = torch.full((B, S, 576), SENTINEL, dtype=torch.bfloat16, device="cuda")
    bt = None
    if is_paged:
        k_base, bt = ref.paged(k_base, gen)
        v_base = torch.full((k_base.shape[0], 64, 576), SENTINEL, dtype=torch.bfloat16, device="cuda")
        k_base.fill_(SENTINEL)
    k_pre = normal(B, T, D, dtype=torch.float32) * 3 + 1
    kv_new = normal(B, T, 576)
    pos = torch.randint(0, S + 5, (B, T), generator=gen, device="cuda").int() if own_pos else None
    q_pe = normal(B, T, H, 64) if H else None
    q_lat = torch.full((B, T, H, 576), SENTINEL, dtype=torch.bfloat16, device="cuda") if H else None
    q_idx = normal(B, T, HI, D) if HI else None
    before = None if q_idx is None else q_idx.clone()
    q_out = None if in_place or q_idx is None else torch.full_like(q_idx, SENTINEL)
    ws = dsa.dsa_cache_append_rope(
        k_pre, kv_new, dsa.Rows(k_base, bt), dsa.Rows(v_base, bt), _i32(start), table, pos=pos,
        n_new=None if n_new is None else _i32(n_new), q_pe=q_pe, q_lat=q_lat, q_idx=q_idx,
        q_idx_out=q_out, kv_style=kv_style, key_style=key_style, eps=EPS)
    assert dsa.read_device_status(ws)[0] == dsa.DSA_OK
    if q_out is None:
        q_out = q_idx
    elif q_idx is not None:
        assert torch.equal(q_idx, before)
    rope = _np(table)
    seen_k = torch.zeros(k_base.shape[:2], dtype=torch.bool)
    for b in range(B):
        n = T if n_new is None else n_new[b]
        for i in range(n):
            row = start[b] + i
            at = (b, row) if bt is None else (int(bt[b, row // 64]), row % 64)
            seen_k[at] = True
            ang = rope[int(pos[b, i]) if own_pos else row]
            x = k_pre[b, i].cpu().numpy()
            mean = x.astype(np.float64).mean()
            v = (x - mean) / math.sqrt(((x - mean) ** 2).mean() + EPS)
            off = layernorm_delta(x, v, EPS)
            v[:64], off[:64] = _turn(v[:64], off[:64], ang, key_style)
            check_bf16_of(_bits(k_base[at]), v, off, f"key {b} {i}")
            v = _np(kv_new[b, i])
            assert torch.equal(v_base[at][:512], kv_new[b, i, :512])
            r, off = _turn(v[512:], np.zeros(64), ang, kv_style)
            check_bf16_of(_bits(v_base[at][512:]), r, off, f"latent row {b} {i}")
            if H:
                r, off = _turn(_np(q_pe[b, i]), np.zeros((H, 64)), ang, kv_style)
                check_bf16_of(_bits(q_lat[b, i, :, 512:]), r, off, f"q_lat {b} {i}")
            if HI:
                r, off = _turn(_np(before[b, i, :, :64]), np.zeros((HI, 64)), ang, key_style)
                check_bf16_of(_bits(q_out[b, i, :, :64]), r, off, f"q_idx {b} {i}")
                assert torch.equal(q_out[b, i, :, 64:], before[b, i, :, 64:])
        if H:
            assert (q_lat[b, n:] == SENTINEL).all()
        if HI:
            assert torch.equal(q_out[b, n:], before[b, n:]) if in_place else (q_out[b, n:] == SENTINEL).all()
    assert (k_base[~seen_k.cuda()] == SENTINEL).all() and (v_base[~seen_k.cuda()] == SENTINEL).all()
    if H:
        assert (q_lat[..., :512] == SENTINEL).all()


def test_append_without_rotation_is_the_plain_append(dsa):
    gen = _gen(5)
    k_pre = torch.randn((2, 9, 128), generator=gen, device="cuda")
    kv_new = torch.randn((2, 9, 576), generator=gen, device="cuda").to(torch.bfloat16)
    stores = [torch.zeros((2, 50, w), dtype=torch.bfloat16, device="cuda") for w in (128, 576, 128, 576)]
    dsa.dsa_cache_append(k_pre, kv_new, dsa.Rows(stores[0]), dsa.Rows(stores[1]), _i32([3, 41]), EPS)
    dsa.dsa_cache_append_rope(k_pre, kv_new, dsa.Rows(stores[2]), dsa.Rows(stores[3]), _i32([3, 41]),
                              _table(50), kv_style=dsa.ROPE_NONE, key_style=dsa.ROPE_NONE, eps=EPS)
    assert torch.equal(stores[0], stores[2]) and torch.equal(stores[1], stores[3])


def test_append_rope_bad_rows_and_positions(dsa):
    """Row 50 does not exist, position 60 is not in the table, n_new is out of range: flagged,
    the rest written."""
    gen = _gen(6)
    k_pre = torch.randn((3, 4, 128), generator=gen, device="cuda")
    kv_new = torch.randn((3, 4, 576), generator=gen, device="cuda").to(torch.bfloat16)
    table = _table(60)

    def run(start, pos=None, n_new=None):
        k = torch.full((3, 50, 128), SENTINEL, dtype=torch.bfloat16, device="cuda")
        v = torch.full((3, 50, 576), SENTINEL, dtype=torch.bfloat16, device="cuda")
        ws = dsa.dsa_cache_append_rope(k_pre, kv_new, dsa.Rows(k), dsa.Rows(v), _i32(start), table,
                                       pos=pos, n_new=n_new)
        return k, v, dsa.read_device_status(ws)[0]

    k0, v0, code = run([0, 10, 46])
    assert code == dsa.DSA_OK
    k, v, code = run([0, 10, 48])
    assert code == dsa.DSA_ERR_BAD_INDEX
    assert torch.equal(k[:2], k0[:2]) and torch.equal(v[:2], v0[:2])
    assert torch.equal(v[2, 48:, :512], kv_new[2, :2, :512]) and (v[2, :48] == SENTINEL).all()
    pos = _i32([[0, 1, 2, 3], [10, 60, 12, -1], [46, 47, 48, 49]])
    k, v, code = run([0, 10, 46], pos=pos)
    assert code == dsa.DSA_ERR_BAD_INDEX
    gone = torch.zeros((3, 50), dtype=torch.bool, device="cuda")
    gone[1, 11] = gone[1, 13] = True
    assert torch.equal(v[~gone], v0[~gone]) and torch.equal(k[~gone], k0[~gone])
    assert (v[gone] == SENTINEL).all() and (k[gone] == SENTINEL).all()
    k, v, code = run([0, 10, 46], n_new=_i32([4, 9, -3]))
    assert code == dsa.DSA_ERR_BAD_INDEX
    assert torch.equal(v[:2], v0[:2]) and (v[2] == SENTINEL).all() and (k[2] == SENTINEL).all()


def test_append_then_tree_then_window(dsa):
    """The operators together, as a decoding step with drafted tokens uses them: append with
    rotation at the tree's depths, then attention over the cache."""
    gen = _gen(7)
    B, T, H, L = 2, 5, 96, [130, 61]
    S = 200
    k = torch.zeros((B, S, 128), dtype=torch.bfloat16, device="cuda")
    kv = torch.randn((B, S, 576), generator=gen, device="cuda").to(torch.bfloat16)
    kv_pool, bt = ref.paged(kv, gen)
    k_pool = torch.zeros((kv_pool.shape[0], 64, 128), dtype=torch.bfloat16, device="cuda")
    rows = dsa.Rows(kv_pool, bt)
    depth = torch.tensor([0, 1, 1, 2, 2], device="cuda")
    masks = torch.tensor([[1, 3, 5, 11, 21]] * B, dtype=torch.int64, device="cuda")
    kl = _i32(L)
    pos = (kl[:, None] + depth).int()
    q_lat = torch.randn((B, T, H, 576), generator=gen, device="cuda").to(torch.bfloat16)
    q_pe = torch.randn((B, T, H, 64), generator=gen, device="cuda").to(torch.bfloat16)
    new = torch.randn((B, T, 576), generator=gen, device="cuda").to(torch.bfloat16)
    ws = dsa.new_workspace(max(dsa.workspace_bytes(dsa.OP_MLA_TREE, B, T, S, H, 0),
                               dsa.workspace_bytes(dsa.OP_MLA_WINDOW, B, 1, S, H, 50)))
    dsa.dsa_cache_append_rope(torch.randn((B, T, 128), generator=gen, device="cuda"), new,
                              dsa.Rows(k_pool, bt), rows, kl, _table(S), pos=pos, q_pe=q_pe,
                              q_lat=q_lat, workspace=ws)
    o, lse = dsa.mla_tree_fwd(q_lat, rows, masks, kl, S, workspace=ws)
    last = q_lat[:, :1].contiguous()
    w, w_lse = dsa.mla_window_fwd(last, rows, kl, kl + 1, 40, 4, S, workspace=ws)
    assert dsa.read_device_status(ws)[0] == dsa.DSA_OK
    for b in range(B):
        cache = ref.logical(kv_pool, bt, b, L[b] + T)
        assert torch.equal(cache[L[b]:, :512], new[b, :, :512].double())
        bits = torch.tensor([[m >> j & 1 for j in range(T)] for m in [1, 3, 5, 11, 21]], device="cuda").bool()
        see = torch.cat([torch.ones((T, L[b]), dtype=torch.bool, device="cuda"), bits], 1)
        r_o, r_lse, o_off, lse_off = ref.forward(q_lat[b], cache, see)
        ref.within(o[b], r_o, o_off, "tree o_lat")
        ref.within(lse[b], r_lse, lse_off, "tree lse")
        n = L[b] + 1
        see = ref.window_sees(torch.tensor([[L[b]]], device="cuda"), torch.arange(n, device="cuda"), 40, 4)
        r_o, r_lse, o_off, lse_off = ref.forward(last[b], cache[:n], see)
        ref.within(w[b], r_o, o_off, "window o_lat")
        ref.within(w_lse[b], r_lse, lse_off, "window lse")


def test_append_rope_in_a_graph(dsa):
    """Captured and replayed with other tokens and places."""
    gen = _gen(8)
    B, T, S = 2, 3, 100
    k, v = (torch.zeros((B, S, w), dtype=torch.bfloat16, device="cuda") for w in (128, 576))
    table, qs = _table(S), _i32([0, 0])
    k_pre = torch.zeros((B, T, 128), device="cuda")
    kv_new, q_pe = (torch.zeros((B, T, w), dtype=torch.bfloat16, device="cuda") for w in (576, 8 * 64))
    q_pe = q_pe.view(B, T, 8, 64)
    q_lat = torch.zeros((B, T, 8, 576), dtype=torch.bfloat16, device="cuda")
    ws = dsa.new_workspace(256)

    def call(k, v, q_lat):
        dsa.dsa_cache_append_rope(k_pre, kv_new, dsa.Rows(k), dsa.Rows(v), qs, table, q_pe=q_pe,
                                  q_lat=q_lat, workspace=ws)

    call(k, v, q_lat)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(k, v, q_lat)
    for start in ([5, 90], [97, 0]):
        qs.copy_(_i32(start))
        k_pre.normal_(generator=gen)
        kv_new.normal_(generator=gen)
        q_pe.normal_(generator=gen)
        other = [x.clone() for x in (k, v, q_lat)]
        graph.replay()
        call(*other)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((k, v, q_lat), other))
    assert dsa.read_device_status(ws)[0] == dsa.DSA_OK


def test_append_rope_beyond_32_bit_offsets(dsa):
    """Caches and queries of more than 2^31 elements: the last rows."""
    gen = _gen(9)
    pages, T, H = 60000, 21000, 96
    v = torch.zeros((pages, 64, 576), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((pages, 64, 128), dtype=torch.bfloat16, device="cuda")
    n = -(-T // 64)
    table = torch.arange(pages - 2 * n, pages, device="cuda", dtype=torch.int32).view(2, n).contiguous()
    q_lat = torch.zeros((2, T, H, 576), dtype=torch.bfloat16, device="cuda")
    assert v.numel() > 2 ** 31 and q_lat.numel() > 2 ** 31
    k_pre = torch.randn((2, T, 128), generator=gen, device="cuda")
    kv_new = torch.randn((2, T, 576), generator=gen, device="cuda").to(torch.bfloat16)
    q_pe = torch.randn((2, T, H, 64), generator=gen, device="cuda").to(torch.bfloat16)
    rope = _table(T)
    ws = dsa.dsa_cache_append_rope(k_pre, kv_new, dsa.Rows(k, table), dsa.Rows(v, table), _i32([0, 0]),
                                   rope, q_pe=q_pe, q_lat=q_lat)
    assert dsa.read_device_status(ws)[0] == dsa.DSA_OK
    got = ref.logical(v, table, 1, T)
    assert torch.equal(got[:, :512], kv_new[1, :, :512].double())
    ang = rope.double()
    x = q_pe[1, -3:].double()
    c, s = ang[-3:, None, :32], ang[-3:, None, 32:]
    want = torch.cat([x[..., :32] * c - x[..., 32:] * s, x[..., 32:] * c + x[..., :32] * s], -1)
    size = (x[..., :32].abs() + x[..., 32:].abs()).repeat(1, 1, 2)
    assert ((q_lat[1, -3:, :, 512:].double() - want).abs() <= want.abs() * ref.HALF + size * 2.0 ** -22).all()
