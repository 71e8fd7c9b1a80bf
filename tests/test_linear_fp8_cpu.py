"""Host-side checks of the FP8 projection path (dsa_rmsnorm_fp8,
dsa_quant_fp8_weight, dsa_linear_fp8): every refusal happens before any launch,
and calls with nothing to do return at once.  CPU only."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
FAKE = P(1 << 20)     # aligned, never dereferenced
OFF8 = P((1 << 20) + 8)
OFF2 = P((1 << 20) + 2)
WS = P(1 << 24)


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_attention_serving_gb300 as m
    return m


def test_rmsnorm_refusals(dsa):
    def call(x=FAKE, r=FAKE, g=FAKE, n=4, hid=1024, eps=1e-5, ro=P(1 << 21), y=P(1 << 22), c=FAKE,
             s=FAKE):
        return dsa.lib.dsa_rmsnorm_fp8(x, r, g, n, hid, eps, ro, y, c, s, None)

    bad, no = dsa.DSA_ERR_INVALID_ARGUMENT, dsa.DSA_ERR_UNSUPPORTED
    for kw in (dict(x=None), dict(g=None), dict(c=None), dict(s=None), dict(n=-1), dict(hid=0),
               dict(hid=-16), dict(eps=-1e-5), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(x=OFF8), dict(r=OFF8), dict(g=OFF8), dict(ro=OFF8), dict(y=OFF8), dict(c=OFF8),
               dict(s=OFF2), dict(r=None),                       # residual_out without a residual
               dict(ro=P(1 << 21), y=P(1 << 21))):               # two outputs in one place
        assert call(**kw) == bad, kw
    for kw in (dict(hid=1000), dict(hid=8), dict(hid=65552), dict(n=1 << 31)):
        assert call(**kw) == no, kw
    # nothing to do: no pointer is looked at
    assert call(x=None, r=None, g=None, n=0, ro=None, y=None, c=None, s=None) == dsa.DSA_OK


def test_quant_weight_refusals(dsa):
    def call(w=FAKE, N=128, K=256, c=FAKE, s=FAKE):
        return dsa.lib.dsa_quant_fp8_weight(w, N, K, c, s, None)

    for kw in (dict(w=None), dict(c=None), dict(s=None), dict(N=0), dict(N=-1), dict(K=0),
               dict(w=OFF8), dict(c=OFF8), dict(s=OFF2)):
        assert call(**kw) == dsa.DSA_ERR_INVALID_ARGUMENT, kw
    for kw in (dict(K=100), dict(N=1 << 30), dict(K=1 << 30), dict(N=(1 << 30) - 1, K=(1 << 30) - 16)):
        assert call(**kw) == dsa.DSA_ERR_UNSUPPORTED, kw


def test_linear_refusals(dsa):
    need = dsa.workspace_bytes(dsa.OP_LINEAR_FP8, 64, 1, 7168, 8192, 0)
    assert need >= 256 and need % 256 == 0

    def call(a=FAKE, sa=FAKE, w=FAKE, sw=FAKE, M=64, N=8192, K=7168, out=FAKE, t=0, ws=WS, n=need):
        return dsa.lib.dsa_linear_fp8(a, sa, w, sw, M, N, K, out, t, ws, n, None)

    for kw in (dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(out=None),
               dict(M=-1), dict(N=0), dict(K=0), dict(t=2), dict(t=-1), dict(a=OFF8), dict(w=OFF8),
               dict(out=OFF8), dict(sa=OFF2), dict(sw=OFF2), dict(ws=None), dict(ws=P((1 << 24) + 8))):
        assert call(**kw) == dsa.DSA_ERR_INVALID_ARGUMENT, kw
    for kw in (dict(K=7160), dict(M=1 << 30), dict(N=1 << 30), dict(K=1 << 30)):
        assert call(**kw) == dsa.DSA_ERR_UNSUPPORTED, kw
    assert call(n=need - 1) == dsa.DSA_ERR_WORKSPACE_TOO_SMALL
    assert call(a=None, sa=None, M=0, out=None, ws=None, n=0) == dsa.DSA_OK


def test_binding_refuses_host_tensors_and_wrong_types(dsa):
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    g = torch.zeros(128, dtype=torch.bfloat16)
    with pytest.raises(dsa.DsaError):
        dsa.dsa_rmsnorm_fp8(x, g)
    with pytest.raises(dsa.DsaError):
        dsa.dsa_quant_fp8_weight(x)
    with pytest.raises(dsa.DsaError):
        dsa.dsa_linear_fp8(x.view(torch.uint8), torch.zeros(4, 2), x.view(torch.uint8), torch.zeros(1, 2))
    with pytest.raises(TypeError):
        dsa.dsa_rmsnorm_fp8([1.0], g)


def test_selftest_refusals(dsa):
    def call(tokens, slices, K=7168, M=64, a=FAKE):
        return dsa.lib.dsa_selftest_linear_fp8(a, FAKE, FAKE, FAKE, M, 8192, K, FAKE, 0, tokens, slices,
                                               WS, 256, None)

    for at in ((0, 2), (1, 1), (16, 0), (16, 7), (16, 17), (96, 12), (128, 16), (256, 1), (-16, 1)):
        assert call(*at) == dsa.DSA_ERR_UNSUPPORTED, at
    assert call(64, 4, K=384) == dsa.DSA_ERR_UNSUPPORTED          # three blocks of K
    assert call(64, 4, K=7160) == dsa.DSA_ERR_UNSUPPORTED
    assert call(64, 4, a=None) == dsa.DSA_ERR_INVALID_ARGUMENT
    assert call(64, 4, M=0) == dsa.DSA_OK


def test_refuse_names_the_operand_and_never_returns(dsa):
    bf, u8, f32 = torch.bfloat16, torch.uint8, torch.float32
    t = lambda dtype, *shape: torch.zeros(shape, dtype=dtype)  # noqa: E731
    good = [(t(bf, 4, 256), (bf,), (4, 256), "x"), (t(u8, 4, 256), (u8,), None, "codes"),
            (t(f32, 4, 2), (bf, f32), (4, 2), "out")]
    with pytest.raises(dsa.DsaError, match="call: operands"):      # nothing to find
        dsa._refuse("call", -1, *good)
    for i, (x, dtypes, shape, name) in enumerate(good):
        wrong = [(x.double(), TypeError), ([1.0], TypeError), (None, TypeError),
                 (torch.zeros(256, 4, dtype=x.dtype).t()[:x.shape[0], :x.shape[1]], dsa.DsaError)]
        if shape is not None:
            wrong.append((x[:2], ValueError))
        for y, error in wrong:
            rules = list(good)
            rules[i] = (y, dtypes, shape, name)
            with pytest.raises(error, match=name):
                dsa._refuse("call", -1, *rules)
    with pytest.raises(dsa.DsaError, match="x must be on cuda:0"):
        dsa._refuse("call", 0, *good)
