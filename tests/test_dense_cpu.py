"""Host-side refusals of dsa_cache_append_rope, mla_tree_fwd, mla_window_fwd and
mla_window_bwd: every one happens before any launch.  CPU only."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
FAKE, OTHER = P(1 << 20), P(1 << 22)     # aligned, never dereferenced
OFF8, OFF2 = P((1 << 20) + 8), P((1 << 20) + 2)
WS = P(1 << 24)


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_attention_serving_gb300 as m
    return m


def _rows(dsa, base=1 << 20, bt=0, stride=128, maxp=0, page=0, npages=0):
    return dsa._Rows(base, stride, bt, maxp, page, npages)


def _refused(call, code, variants):
    for kw in variants:
        assert call(**kw) == code, kw


def test_append_rope_refusals(dsa):
    def call(k_pre=FAKE, kv_new=FAKE, kr=None, vr=None, qs=FAKE, rope=FAKE, n_pos=10, pos=None,
             n_new=None, q_pe=FAKE, q_lat=OTHER, H=96, q_idx=FAKE, q_out=OTHER, HI=64, B=1, T=1,
             D=128, ks=1, kk=1, eps=1e-5, ws=WS, n=256):
        kr, vr = kr or _rows(dsa), vr or _rows(dsa)
        return dsa.lib.dsa_cache_append_rope(k_pre, kv_new, kr, vr, qs, rope, n_pos, pos, n_new, q_pe,
                                             q_lat, H, q_idx, q_out, HI, B, T, D, ks, kk, eps, ws, n,
                                             None)

    bad, no = dsa.DSA_ERR_INVALID_ARGUMENT, dsa.DSA_ERR_UNSUPPORTED
    _refused(call, bad, [dict(k_pre=None), dict(kv_new=None), dict(qs=None), dict(rope=None),
                         dict(q_pe=None), dict(q_lat=None), dict(q_idx=None), dict(q_out=None),
                         dict(k_pre=OFF8), dict(kv_new=OFF8), dict(rope=OFF8), dict(q_pe=OFF8),
                         dict(q_lat=OFF8), dict(q_idx=OFF8), dict(q_out=OFF8), dict(qs=OFF2),
                         dict(pos=OFF2), dict(n_new=OFF2), dict(n_pos=0), dict(H=0), dict(HI=0),
                         dict(B=0), dict(T=0), dict(T=-1), dict(ks=3), dict(kk=-1), dict(eps=-1.0),
                         dict(eps=float("nan")), dict(eps=float("inf")), dict(ws=None), dict(ws=OFF8),
                         dict(kr=_rows(dsa, base=0)), dict(vr=_rows(dsa, base=(1 << 20) + 8)),
                         dict(vr=_rows(dsa, bt=1 << 20, page=64, maxp=0, npages=4))])
    _refused(call, no, [dict(D=96), dict(H=1025), dict(HI=1025), dict(B=1 << 13, T=1 << 12),
                        dict(kr=_rows(dsa, bt=1 << 20, page=32, maxp=1, npages=4))])
    assert call(n=255) == dsa.DSA_ERR_WORKSPACE_TOO_SMALL


def _dense_variants(bad, no, dsa, pos="pos0"):
    return ([dict(q=None), dict(o=None), {pos: None}, dict(kv=_rows(dsa, base=0)), dict(q=OFF8),
             dict(o=OFF8), dict(lse=OFF2), {pos: OFF2}, dict(lim=OFF2), dict(B=0), dict(T=0), dict(H=0),
             dict(S=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
             dict(scale=float("inf")), dict(ws=None), dict(ws=OFF8), dict(S=129),
             dict(kv=_rows(dsa, base=(1 << 20) + 8))],
            [dict(H=129), dict(B=1 << 25, T=1, H=64), dict(kv=_rows(dsa, stride=1 << 31))])


def test_tree_refusals(dsa):
    def call(q=FAKE, kv=None, tree=FAKE, pos0=FAKE, lim=None, B=1, T=4, H=96, S=128, scale=0.1,
             o=FAKE, lse=FAKE, ws=WS, n=1 << 40):
        return dsa.lib.mla_tree_fwd(q, kv or _rows(dsa), tree, pos0, lim, B, T, H, S, scale, o, lse, ws, n,
                                    None)

    bad, no = _dense_variants(dsa.DSA_ERR_INVALID_ARGUMENT, dsa.DSA_ERR_UNSUPPORTED, dsa)
    paged = dict(bt=1 << 20, stride=0, maxp=2, npages=4)
    _refused(call, dsa.DSA_ERR_INVALID_ARGUMENT,
             bad + [dict(tree=None), dict(tree=P((1 << 20) + 4)), dict(kv=_rows(dsa, page=64, **paged), S=129)])
    _refused(call, dsa.DSA_ERR_UNSUPPORTED, no + [dict(T=65), dict(kv=_rows(dsa, page=128, **paged))])
    assert call(n=255) == dsa.DSA_ERR_WORKSPACE_TOO_SMALL


def test_window_refusals(dsa):
    def call(q=FAKE, kv=None, pos0=FAKE, lim=FAKE, B=1, T=4, H=96, w=64, f=4, S=128, scale=0.1, o=FAKE,
             lse=FAKE, ws=WS, n=1 << 40):
        return dsa.lib.mla_window_fwd(q, kv or _rows(dsa), pos0, lim, B, T, H, w, f, S, scale, o, lse, ws,
                                      n, None)

    bad, no = _dense_variants(dsa.DSA_ERR_INVALID_ARGUMENT, dsa.DSA_ERR_UNSUPPORTED, dsa)
    _refused(call, dsa.DSA_ERR_INVALID_ARGUMENT, bad + [dict(lim=None), dict(w=-1), dict(f=-1)])
    _refused(call, dsa.DSA_ERR_UNSUPPORTED, no)
    assert call(n=255) == dsa.DSA_ERR_WORKSPACE_TOO_SMALL


def test_window_bwd_refusals(dsa):
    def call(q=FAKE, kv=None, pos0=FAKE, lim=FAKE, B=1, T=4, H=96, w=64, f=4, S=128, scale=0.1, o=FAKE,
             lse=FAKE, d_o=FAKE, dq=FAKE, dkv=FAKE, ws=WS, n=1 << 40):
        return dsa.lib.mla_window_bwd(q, kv or _rows(dsa), pos0, lim, B, T, H, w, f, S, scale, o, lse, d_o,
                                      dq, dkv, ws, n, None)

    bad, no = _dense_variants(dsa.DSA_ERR_INVALID_ARGUMENT, dsa.DSA_ERR_UNSUPPORTED, dsa)
    _refused(call, dsa.DSA_ERR_INVALID_ARGUMENT,
             bad + [dict(lim=None), dict(w=-1), dict(f=-1), dict(lse=None), dict(d_o=None), dict(dq=None),
                    dict(dkv=None), dict(d_o=OFF8), dict(dq=OFF8), dict(dkv=OFF8)])
    _refused(call, dsa.DSA_ERR_UNSUPPORTED,
             no + [dict(kv=_rows(dsa, bt=1 << 20, page=64, maxp=2, npages=4))])
    assert call(n=255) == dsa.DSA_ERR_WORKSPACE_TOO_SMALL


def test_workspace_sizes(dsa):
    for op in (dsa.OP_MLA_TREE, dsa.OP_MLA_WINDOW, dsa.OP_MLA_WINDOW_BWD):
        for B, T, S, H, span in ((1, 1, 1, 1, 1), (1, 1, 131072, 96, 0), (64, 1, 9001, 96, 516),
                                 (2, 8192, 8192, 96, 1040), (3, 301, 301, 8, 80), (1, 64, 70, 128, 5)):
            n = dsa.workspace_bytes(op, B, T, S, H, span)
            assert n >= 256 and n % 256 == 0 and n < 1 << 34
        assert dsa.workspace_bytes(op, 0, 1, 1, 1, 1) == 256
        assert dsa.workspace_bytes(op, 1, 1, 1, 0, 1) == 256


def test_binding_refuses_cpu_tensors(dsa):
    q = torch.zeros((1, 1, 8, 576), dtype=torch.bfloat16)
    with pytest.raises(dsa.DsaError):
        dsa.mla_tree_fwd(q, None, None, None, 64)
    with pytest.raises(dsa.DsaError):
        dsa.mla_window_fwd(q, None, None, None, 4, 0, 64)
    with pytest.raises(dsa.DsaError):
        dsa.mla_window_bwd(q, None, None, None, 4, 0, 64, None, None, None)
    with pytest.raises(dsa.DsaError):
        dsa.dsa_cache_append_rope(torch.zeros((1, 1, 128)), None, None, None, None, None)
    with pytest.raises(TypeError):
        dsa.mla_tree_fwd(None, None, None, None, 64)
