"""GPU parity of the FP8 projection path (dsa_rmsnorm_fp8, dsa_quant_fp8_weight,
dsa_linear_fp8) against plain 64-bit computations, with bounds derived from the
number of FP32 operations:

* norm: a row's sum of squares has at most 64 sequential additions per thread
  and 11 tree levels, all of one sign, so 1/sqrt of it is off by at most about
  40 * 2^-24 and y by a few more: 2^-18 covers it (Y_REL).  Codes must be the
  E4M3 rounding of some value within that of y / scale.
* weight: every operation is one correctly rounded FP32 operation, so codes and
  scales are equal bit for bit.
* product: within a block the tensor core adds 128 exact products (each addition
  off by at most 2^-23 of the running magnitude, truncation allowed), then one
  FP32 product of scales and one FMA per block: (128 + blocks + 2) * 2^-23 of the
  sum of magnitudes, plus half a step of out's type (finfo.eps / 2).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import bf, check_gate_rows, check_indexer_rows, check_mla_rows, i32, to_u16
from parity import check_bf16_of
from workloads import CONFIGS, bf16_to_f32

pytestmark = pytest.mark.gpu

EPS = 1e-5
Y_REL = 2.0 ** -18
FLOOR = np.float32(2.0 ** -100) / np.float32(448)


@pytest.fixture(scope="module")
def dsa():
    import sparse_attention_serving_gb300 as m
    return m


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(seed, n, width, scale=1.0):
    """BF16 rows whose blocks differ in size by orders of magnitude."""
    g = _gen(seed)
    x = torch.randn((n, width), generator=g, device="cuda") * scale
    x *= torch.exp2(torch.randint(-6, 7, (n, -(-width // 128)), generator=g, device="cuda").float()
                    ).repeat_interleave(128, 1)[:, :width]
    return x.to(torch.bfloat16)


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------

def _check_norm(x, residual, gain, eps, codes, scale, residual_out, y, what):
    """x, residual, gain: float64 CPU arrays; the rest as the GPU returned it."""
    h = x if residual is None else x + residual
    hid = h.shape[1]
    v = h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * gain
    if residual_out is not None:
        check_bf16_of(to_u16(residual_out), h, 2.0 ** -24 * np.abs(h), f"{what} residual_out")
    if y is not None:
        check_bf16_of(to_u16(y), v, Y_REL * np.abs(v), f"{what} y")
    nb = -(-hid // 128)
    full = np.zeros((h.shape[0], nb * 128))
    full[:, :hid] = np.abs(v)
    top = full.reshape(-1, nb, 128).max(2)
    want = np.maximum(top, 2.0 ** -100) / 448
    s = scale.cpu().numpy().astype(np.float64)
    assert s.shape == want.shape
    # one division on top of y's error
    assert np.all(np.abs(s - want) <= (Y_REL + 2.0 ** -24) * want), f"{what} scale"
    # the codes, by the GPU's own scales: the reciprocal and the product add 2^-24 each
    t = v / np.repeat(s, 128, axis=1)[:, :hid]
    d = (Y_REL + 2.0 ** -22) * np.abs(t)
    got = oracle.e4m3_decode(codes.cpu().numpy())
    lo = oracle.e4m3_decode(oracle.e4m3_encode((t - d).astype(np.float32)))
    hi = oracle.e4m3_decode(oracle.e4m3_encode((t + d).astype(np.float32)))
    bad = ~((got >= lo) & (got <= hi))
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], t[bad][:4])


@pytest.mark.parametrize("n,hid", [(1, 16), (3, 112), (1, 128), (5, 144), (37, 1024), (2, 1040),
                                   (9, 7168), (3, 7184), (2, 16384), (1, 65536), (300, 256)])
@pytest.mark.parametrize("with_residual,with_y", [(True, True), (False, False)])
def test_norm(dsa, n, hid, with_residual, with_y):
    x = _rows(n * 7 + hid, n, hid)
    x[-1, hid // 2:] = 0                       # blocks of zeros (the whole row when hid is 16)
    r = _rows(n * 7 + hid + 1, n, hid) if with_residual else None
    if r is not None:
        r[-1, hid // 2:] = 0
    gain = (1 + 0.1 * torch.randn(hid, generator=_gen(5), device="cuda")).to(torch.bfloat16)
    # one more row behind the last of every output stays as it was
    bufs = [torch.full((n + 1, hid), 0x5A, dtype=torch.uint8, device="cuda"),
            torch.full((n + 1, -(-hid // 128)), 7.5, device="cuda"),
            torch.full((n + 1, hid), 7.5, dtype=torch.bfloat16, device="cuda"),
            torch.full((n + 1, hid), 7.5, dtype=torch.bfloat16, device="cuda")]
    codes, scale, ro, y = dsa.dsa_rmsnorm_fp8(
        x, gain, residual=r, eps=EPS, codes=bufs[0][:n], scale=bufs[1][:n],
        residual_out=bufs[2][:n] if with_residual else None, y=bufs[3][:n] if with_y else None)
    d = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    _check_norm(d(x), d(r), d(gain), EPS, codes, scale, ro, y, f"{n}x{hid}")
    assert (bufs[0][n] == 0x5A).all() and all((b[n] == 7.5).all() for b in bufs[1:])
    if not with_residual:
        assert ro is None and (bufs[2] == 7.5).all()
    if not with_y:
        assert y is None and (bufs[3] == 7.5).all()


def test_norm_zero_rows_and_no_rows(dsa):
    x = torch.zeros((3, 1040), dtype=torch.bfloat16, device="cuda")
    gain = torch.ones(1040, dtype=torch.bfloat16, device="cuda")
    codes, scale, ro, y = dsa.dsa_rmsnorm_fp8(x, gain, residual=x, want_y=True)
    assert (codes == 0).all() and (ro == 0).all() and (y == 0).all()
    assert (scale.cpu().numpy() == FLOOR).all()
    # eps = 0 on a row of zeros is 0 * inf: NaN, as the formula says
    codes, scale, _, y = dsa.dsa_rmsnorm_fp8(x, gain, eps=0.0, want_y=True)
    assert torch.isnan(y).all() and torch.isnan(scale).all()
    codes, scale, ro, y = dsa.dsa_rmsnorm_fp8(x[:0], gain, residual=x[:0], want_y=True)
    assert codes.shape == (0, 1040) and scale.shape == (0, 9) and ro.shape == y.shape == (0, 1040)


def test_norm_non_finite_values_stay_in_their_row(dsa):
    x = _rows(3, 6, 512)
    clean = dsa.dsa_rmsnorm_fp8(x, torch.ones(512, dtype=torch.bfloat16, device="cuda"), want_y=True)
    gain = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    x[1, 300] = float("nan")
    x[3, 10] = float("inf")
    codes, scale, _, y = dsa.dsa_rmsnorm_fp8(x, gain, want_y=True)
    # NaN: the whole row; infinity: 1/sqrt is 0, so NaN at its place and zeros elsewhere
    assert torch.isnan(y[1]).all() and torch.isnan(scale[1]).all()
    assert torch.isnan(y[3, 10]) and torch.isnan(scale[3, 0])
    assert (y[3, 128:] == 0).all() and (scale[3, 1:] == float(FLOOR)).all()
    keep = [0, 2, 4, 5]
    for a, b in zip(clean, (codes, scale, None, y)):
        if b is not None:
            assert torch.equal(a[keep], b[keep])


def test_norm_in_place_and_leading_dims(dsa):
    x, r = _rows(21, 40, 1024), _rows(22, 40, 1024)
    gain = (1 + 0.1 * torch.randn(1024, generator=_gen(5), device="cuda")).to(torch.bfloat16)
    want = dsa.dsa_rmsnorm_fp8(x, gain, residual=r, want_y=True)
    x1, r1 = x.clone().view(4, 10, 1024), r.clone().view(4, 10, 1024)
    codes, scale, ro, y = dsa.dsa_rmsnorm_fp8(x1, gain, residual=r1, residual_out=r1, y=x1)
    assert ro is r1 and y is x1 and codes.shape == (4, 10, 1024) and scale.shape == (4, 10, 8)
    for a, b in zip(want, (codes, scale, ro, y)):
        assert torch.equal(a.flatten(), b.flatten())


# ---------------------------------------------------------------------------
# weight
# ---------------------------------------------------------------------------

def _quant_weight_ref(w):
    """w float32 [N,K] -> codes, scales, in float32 operations."""
    N, K = w.shape
    nb, kb = -(-N // 128), -(-K // 128)
    full = np.zeros((nb * 128, kb * 128), np.float32)
    full[:N, :K] = np.abs(w)
    top = full.reshape(nb, 128, kb, 128).max((1, 3))
    scale = np.maximum(top, np.float32(2.0 ** -100)) / np.float32(448)
    inv = np.float32(1) / scale
    t = w * np.repeat(np.repeat(inv, 128, 0), 128, 1)[:N, :K]
    return oracle.e4m3_encode(t), scale


@pytest.mark.parametrize("N,K", [(1, 16), (128, 128), (129, 144), (100, 4096), (576, 7168), (1001, 1040)])
def test_quant_weight(dsa, N, K):
    w = _rows(N + K, N, K, 0.02)
    w[:, K // 2:] *= 0.25
    w[N // 2:, :16] = 0
    if N > 128:
        w[128:, :] = 0                                        # whole blocks of zeros
    cb = torch.full((N + 1, K), 0x5A, dtype=torch.uint8, device="cuda")
    codes, scale = dsa.dsa_quant_fp8_weight(w, codes=cb[:N])
    ec, es = _quant_weight_ref(bf16_to_f32(to_u16(w)))
    assert np.array_equal(scale.cpu().numpy(), es)
    assert np.array_equal(codes.cpu().numpy(), ec)
    assert (cb[N] == 0x5A).all()


def test_quant_weight_non_finite_values_stay_in_their_block(dsa):
    w = _rows(9, 256, 384, 0.02)
    clean, cs = dsa.dsa_quant_fp8_weight(w)
    w[5, 130] = float("nan")
    w[200, 300] = float("inf")
    codes, scale = dsa.dsa_quant_fp8_weight(w)
    assert torch.isnan(scale[0, 1]) and torch.isinf(scale[1, 2])
    v = codes.view(torch.float8_e4m3fn).float()
    assert torch.isnan(v[:128, 128:256]).all() and torch.isnan(v[200, 300])
    same = torch.ones((2, 3), dtype=torch.bool)
    same[0, 1] = same[1, 2] = False
    assert torch.equal(scale.cpu()[same], cs.cpu()[same])
    mask = same.repeat_interleave(128, 0).repeat_interleave(128, 1)
    assert torch.equal(codes.cpu()[mask], clean.cpu()[mask])


# ---------------------------------------------------------------------------
# product
# ---------------------------------------------------------------------------

def _operands(dsa, seed, M, N, K):
    a = _rows(seed, M, K)
    if M > 2:
        a[M // 2] = 0                                          # a padded token
    pad = -K % 128
    full = torch.nn.functional.pad(a, (0, pad)).view(M, -1, 128)
    c, s = dsa.dsa_quant_fp8(full.contiguous())
    codes = c.view(M, -1)[:, :K].contiguous()
    w_codes, w_scale = dsa.dsa_quant_fp8_weight(_rows(seed + 1, N, K, 0.02))
    return codes, s, w_codes, w_scale


def _linear_ref(codes, scale, w_codes, w_scale):
    """out and the sum of magnitudes, in 64 bits."""
    K, N = codes.shape[-1], w_codes.shape[0]
    col = torch.arange(K, device="cuda") // 128
    row = torch.arange(N, device="cuda") // 128
    a = codes.view(torch.float8_e4m3fn).double() * scale.double()[:, col]
    w = w_codes.view(torch.float8_e4m3fn).double() * w_scale.double()[row][:, col]
    return a @ w.t(), a.abs() @ w.abs().t()


def _check_linear(out, ref, mag, K, what):
    half = torch.finfo(out.dtype).eps / 2
    tol = (128 + -(-K // 128) + 2) * 2.0 ** -23 * mag * (1 + half) + half * ref.abs()
    err = (out.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist(),
                           float((err / tol.clamp(min=1e-300)).max()))


SIZES = [(1, 1, 16), (1, 8, 128), (1, 128, 7168), (2, 129, 144), (1, 8192, 1024), (3, 576, 112),
         (7, 1000, 2064), (8, 300, 256), (9, 1001, 1040), (16, 128, 7168), (17, 4608, 1024),
         (32, 576, 3584), (33, 64, 12288), (64, 256, 2048), (65, 7, 512), (100, 777, 1040),
         (127, 1024, 1024), (128, 1024, 1024), (129, 130, 272), (200, 512, 4096), (256, 576, 7168),
         (257, 255, 400), (300, 257, 1024), (512, 1001, 640), (777, 1001, 1040), (1000, 640, 7168),
         (1025, 1300, 144), (2048, 576, 896), (2500, 2305, 528), (4097, 520, 1024),
         (4100, 1304, 272), (5000, 1000, 2064), (2049, 2564, 144),
         (64, 128, 7168), (400, 256, 7168), (2048, 130, 7168), (96, 1024, 2048), (300, 8192, 512)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear(dsa, M, N, K, dtype):
    codes, scale, w_codes, w_scale = _operands(dsa, M + N + K, M, N, K)
    ws = dsa.new_workspace(dsa.workspace_bytes(dsa.OP_LINEAR_FP8, M, 1, K, N, 0))
    buf = torch.full((M * N + 64,), 7.5, dtype=dtype, device="cuda")
    out = dsa.dsa_linear_fp8(codes, scale, w_codes, w_scale, out=buf[:M * N].view(M, N), workspace=ws)
    assert dsa.read_device_status(ws)[0] == dsa.DSA_OK
    ref, mag = _linear_ref(codes, scale, w_codes, w_scale)
    _check_linear(out, ref, mag, K, f"{M}x{N}x{K}")
    assert (buf[M * N:] == 7.5).all()                          # what lies behind the last row stays
    # equal calls give equal bits
    again = dsa.dsa_linear_fp8(codes, scale, w_codes, w_scale, out_dtype=dtype, workspace=ws)
    assert torch.equal(again, out)


def test_linear_no_rows_and_leading_dims(dsa):
    codes, scale, w_codes, w_scale = _operands(dsa, 4, 24, 130, 272)
    want = dsa.dsa_linear_fp8(codes, scale, w_codes, w_scale)
    got = dsa.dsa_linear_fp8(codes.view(2, 12, 272), scale.view(2, 12, 3), w_codes, w_scale)
    assert got.shape == (2, 12, 130) and torch.equal(got.view(24, 130), want)
    one = dsa.dsa_linear_fp8(codes[3], scale[3], w_codes, w_scale)
    assert one.shape == (130,)
    ref, mag = _linear_ref(codes[3:4], scale[3:4], w_codes, w_scale)
    _check_linear(one[None], ref, mag, 272, "one row")
    none = dsa.dsa_linear_fp8(codes[:0], scale[:0], w_codes, w_scale)
    assert none.shape == (0, 130)


def _repeats(t, period):
    """Row i + period equals row i, to the last row."""
    assert torch.equal(t[period:].view(torch.uint8), t[:-period].view(torch.uint8))


def test_norm_and_weight_offsets_beyond_31_bits(dsa):
    n, hid, period = 300_032, 7168, 1024                       # 2.15e9 values
    few = _rows(5, period, hid)
    x = few.repeat(n // period, 1)
    gain = torch.ones(hid, dtype=torch.bfloat16, device="cuda")
    codes, scale, h, y = dsa.dsa_rmsnorm_fp8(x, gain, residual=x, want_y=True)
    first = dsa.dsa_rmsnorm_fp8(few, gain, residual=few, want_y=True)
    for got, want in zip((codes, scale, h, y), first):
        assert torch.equal(got[:period], want)
        _repeats(got, period)
    del h, y, codes, scale
    codes, scale = dsa.dsa_quant_fp8_weight(x)
    want_codes, want_scale = dsa.dsa_quant_fp8_weight(few)
    assert torch.equal(codes[:period], want_codes) and torch.equal(scale[:period // 128], want_scale)
    _repeats(codes, period)
    _repeats(scale, period // 128)


@pytest.mark.parametrize("M,N,K,dtype", [
    (270_001, 8192, 144, torch.bfloat16),                      # out: TMA and, with odd rows, plain
    (270_001, 8193, 144, torch.bfloat16), (270_001, 8194, 144, torch.float32),
    (300_001, 128, 7168, torch.float32),                       # codes
    (3, 300_032, 7168, torch.bfloat16), (300, 300_032, 7168, torch.bfloat16)])   # weight
def test_linear_offsets_beyond_31_bits(dsa, M, N, K, dtype):
    period = 1024
    m, n = min(M, period), N if N < 10_000 else period
    codes, scale, w_codes, w_scale = _operands(dsa, 6, m, n, K)
    ref, mag = _linear_ref(codes, scale, w_codes, w_scale)
    if M > m:
        i = torch.arange(M, device="cuda") % period
        codes, scale = codes[i], scale[i]
    if N > n:
        w_codes, w_scale = w_codes.repeat(N // n, 1), w_scale.repeat(N // n, 1)
    ws = dsa.new_workspace(dsa.workspace_bytes(dsa.OP_LINEAR_FP8, M, 1, K, N, 0))
    out = dsa.dsa_linear_fp8(codes, scale, w_codes, w_scale, out_dtype=dtype, workspace=ws)
    assert dsa.read_device_status(ws)[0] == dsa.DSA_OK
    _check_linear(out[:m, :n], ref, mag, K, f"{M}x{N}x{K}")
    if M > m:
        _repeats(out, period)
    if N > n:
        _repeats(out.t().contiguous(), n)


@pytest.mark.parametrize("M", [2, 40, 500])
def test_linear_non_finite_values_stay_in_their_row_and_block(dsa, M):
    codes, scale, w_codes, w_scale = _operands(dsa, M, M, 400, 1040)
    clean = dsa.dsa_linear_fp8(codes, scale, w_codes, w_scale, out_dtype=torch.float32)
    codes, scale, w_codes, w_scale = (t.clone() for t in (codes, scale, w_codes, w_scale))
    scale[M - 1, 2] = float("nan")
    codes[0, 700] = 0x7F                                       # a NaN code
    w_codes[17, 1039] = 0xFF
    w_scale[2, 8] = float("nan")
    out = dsa.dsa_linear_fp8(codes, scale, w_codes, w_scale, out_dtype=torch.float32)
    nan = torch.zeros((M, 400), dtype=torch.bool, device="cuda")
    nan[M - 1] = nan[0] = True
    nan[:, 17] = True
    nan[:, 256:384] = True
    assert torch.equal(torch.isnan(out), nan)
    assert torch.equal(out[~nan], clean[~nan])


def test_linear_on_another_stream_and_without_a_workspace(dsa):
    codes, scale, w_codes, w_scale = _operands(dsa, 8, 70, 600, 1040)
    want = dsa.dsa_linear_fp8(codes, scale, w_codes, w_scale)
    x = _rows(2, 70, 1040)
    gain = torch.ones(1040, dtype=torch.bfloat16, device="cuda")
    wn = dsa.dsa_rmsnorm_fp8(x, gain, residual=x, want_y=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = dsa.dsa_linear_fp8(codes, scale, w_codes, w_scale, stream=side)
    gn = dsa.dsa_rmsnorm_fp8(x, gain, residual=x, want_y=True, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    for a, b in zip(wn, gn):
        assert torch.equal(a, b)


@pytest.mark.parametrize("M", [1, 96, 5000])
def test_calls_in_a_row_see_each_other(dsa, M):
    """Kernels on one stream may start while the one before finishes: what a call
    reads is the call's before, and what it overwrites has been read."""
    hid = N = 1040
    gain = (1 + 0.1 * torch.randn(hid, generator=_gen(5), device="cuda")).to(torch.bfloat16)
    weights = [dsa.dsa_quant_fp8_weight(_rows(40 + k, N, hid, 0.03)) for k in range(2)]
    w_bf = [_rows(40 + k, N, hid, 0.03) for k in range(2)]
    ws = dsa.new_workspace(256)

    def run(sync):
        x, h = _rows(50, M, hid), _rows(51, M, hid)
        codes = torch.empty((M, hid), dtype=torch.uint8, device="cuda")
        scale = torch.empty((M, 9), device="cuda")
        wc, wsc = torch.empty_like(weights[0][0]), torch.empty_like(weights[0][1])
        seen = []
        for k in range(40):
            wait = torch.cuda.synchronize if sync else (lambda: None)
            dsa.dsa_rmsnorm_fp8(x, gain, residual=h, codes=codes, scale=scale, residual_out=h, y=x)
            wait()
            dsa.dsa_quant_fp8_weight(w_bf[k % 2], codes=wc, scale=wsc)
            wait()
            dsa.dsa_linear_fp8(codes, scale, wc, wsc, out=x, workspace=ws)
            wait()
            if k % 8 == 7:
                seen.append((x.clone(), h.clone(), codes.clone(), scale.clone()))
        torch.cuda.synchronize()
        return seen

    for a, b in zip(run(True), run(False)):
        for s, t in zip(a, b):
            assert torch.equal(s, t)


def test_two_streams_at_once(dsa):
    cases = [_operands(dsa, 60, 2500, 2304, 1040), _operands(dsa, 61, 24, 1024, 7168),
             _operands(dsa, 62, 700, 576, 2064)]
    want = [dsa.dsa_linear_fp8(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    spaces = [dsa.new_workspace(256) for _ in cases]
    outs = [[torch.empty_like(w) for _ in range(10)] for w in want]
    torch.cuda.synchronize()
    for k in range(10):
        for c, s, ws, o in zip(cases, streams, spaces, outs):
            dsa.dsa_linear_fp8(*c, out=o[k], workspace=ws, stream=s)
    torch.cuda.synchronize()
    for w, o, ws in zip(want, outs, spaces):
        assert all(torch.equal(w, t) for t in o)
        assert dsa.read_device_status(ws)[0] == dsa.DSA_OK


def test_binding_refusals_on_device(dsa):
    codes, scale, w_codes, w_scale = _operands(dsa, 8, 6, 200, 256)
    lin = dsa.dsa_linear_fp8
    with pytest.raises(ValueError):
        lin(codes[:, :128].contiguous(), scale, w_codes, w_scale)
    with pytest.raises(ValueError):
        lin(codes, scale[:, :1].contiguous(), w_codes, w_scale)
    with pytest.raises(ValueError):
        lin(codes, scale, w_codes, w_scale[:1])
    with pytest.raises(TypeError):
        lin(codes, scale.half(), w_codes, w_scale)
    with pytest.raises(TypeError):
        lin(codes, scale, w_codes, w_scale, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        lin(codes, scale, w_codes, w_scale, out=torch.empty((6, 201), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(dsa.DsaError):                          # a strided view
        lin(codes[::2], scale[::2].contiguous(), w_codes, w_scale)
    with pytest.raises(dsa.DsaError):                          # codes off a 16-byte boundary
        lin(torch.zeros(6 * 256 + 1, dtype=torch.uint8, device="cuda")[1:].view(6, 256), scale,
            w_codes, w_scale)
    with pytest.raises(dsa.DsaError):
        lin(codes, scale, w_codes.cpu(), w_scale)
    with pytest.raises(TypeError):
        lin(codes, scale, [1], w_scale)
    with pytest.raises(TypeError):
        lin(codes, scale, w_codes, w_scale, workspace=256)
    with pytest.raises(dsa.DsaError):                          # a workspace without its header
        lin(codes, scale, w_codes, w_scale, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    gain = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        dsa.dsa_rmsnorm_fp8(x, gain[:128].contiguous())
    with pytest.raises(ValueError):
        dsa.dsa_rmsnorm_fp8(x, gain, residual=x[:2])
    with pytest.raises(TypeError):
        dsa.dsa_rmsnorm_fp8(x.float(), gain)
    with pytest.raises(dsa.DsaError):
        dsa.dsa_rmsnorm_fp8(x[:, :248].contiguous(), gain[:248])
    with pytest.raises(dsa.DsaError):
        dsa.dsa_rmsnorm_fp8(x, gain, residual_out=torch.empty_like(x))


def test_sizes_beyond_32_bits_are_refused(dsa):
    """A size whose low 32 bits are a supported one (2^32 + 16 as 16).  The sizes are
    looked at first, so views of a few bytes stand for the large arrays."""
    big = (1 << 32) + 16
    few = lambda shape, dtype=torch.uint8: torch.zeros(  # noqa: E731
        (1,) * len(shape), dtype=dtype, device="cuda").expand(shape)
    calls = [lambda: dsa.dsa_rmsnorm_fp8(few((1, big), torch.bfloat16), few((big,), torch.bfloat16)),
             lambda: dsa.dsa_quant_fp8_weight(few((1, big), torch.bfloat16)),
             lambda: dsa.dsa_quant_fp8_weight(few((big, 16), torch.bfloat16))]
    for m, n, k in ((1, 1, big), (big, 1, 16), (1, big, 16)):
        calls.append(lambda m=m, n=n, k=k: dsa.dsa_linear_fp8(
            few((m, k)), few((m, -(-k // 128)), torch.float32), few((n, k)),
            few((-(-n // 128), -(-k // 128)), torch.float32)))
    for call in calls:
        with pytest.raises(dsa.DsaError) as e:
            call()
        assert e.value.code == dsa.DSA_ERR_UNSUPPORTED


# ---------------------------------------------------------------------------
# the path as a layer uses it
# ---------------------------------------------------------------------------

def _layer(dsa, cfg, x, residual, gain, W, caches, ws, W_g, W_uv, kv_len):
    """residual + norm -> projections -> append -> indexer -> MLA -> gate -> output
    projection, all on the current stream."""
    B, T = x.shape[:2]
    codes, scale, residual, y = dsa.dsa_rmsnorm_fp8(x, gain, residual=residual, want_y=True)
    lin = lambda name, dt=torch.bfloat16: dsa.dsa_linear_fp8(  # noqa: E731
        codes, scale, *W[name], out_dtype=dt, workspace=ws)
    q_idx = lin("q_idx").view(B, T, cfg.H_I, cfg.D_I)
    w = lin("w")
    k_pre = lin("k_pre", torch.float32)
    kv_new = lin("kv")
    q_lat = lin("q_lat").view(B, T, cfg.H, 576)
    q_start = torch.zeros(B, dtype=torch.int32, device="cuda")
    k_rows, kv_rows = (dsa.Rows(c) for c in caches)
    dsa.dsa_cache_append(k_pre, kv_new, k_rows, kv_rows, q_start, workspace=ws)
    idx = dsa.dsa_indexer_topk(q_idx, w, k_rows, q_start, kv_len, cfg.topk, T, workspace=ws)
    o, lse = dsa.sparse_mla_fwd(q_lat, kv_rows, idx, q_start, kv_len, T, cfg.scale, workspace=ws)
    gated = dsa.mla_gate_apply(y.view(B * T, -1), W_g, o.view(B * T, cfg.H, 512), W_uv, workspace=ws)
    oc, os = dsa.dsa_quant_fp8(gated.view(B * T, cfg.H, 128))
    out = dsa.dsa_linear_fp8(oc.view(B * T, -1), os, *W["o"], workspace=ws)
    return dict(codes=codes, scale=scale, residual=residual, y=y, q_idx=q_idx, w=w, k_pre=k_pre,
                kv_new=kv_new, q_lat=q_lat, idx=idx, o=o, lse=lse, gated=gated, oc=oc, os=os, out=out)


def test_layer_around_the_step(dsa):
    cfg = CONFIGS["tiny"]
    B, T, hid = cfg.B, cfg.T, cfg.hid
    g = _gen(77)
    rnd = lambda *s, k=1.0: (torch.randn(s, generator=g, device="cuda") * k).to(torch.bfloat16)  # noqa: E731
    x, residual, gain = rnd(B, T, hid), rnd(B, T, hid), 1 + rnd(hid, k=0.1)
    # fan-in scaling: projections of unit variance, as the step's inputs have
    widths = dict(q_idx=cfg.H_I * cfg.D_I, w=cfg.H_I, k_pre=cfg.D_I, kv=576, q_lat=cfg.H * 576)
    W = {n: dsa.dsa_quant_fp8_weight(rnd(N, hid, k=hid ** -0.5)) for n, N in widths.items()}
    W["o"] = dsa.dsa_quant_fp8_weight(rnd(hid, cfg.H * 128, k=(cfg.H * 128) ** -0.5))
    W_g, W_uv = rnd(cfg.H * 128, hid, k=0.02), rnd(cfg.H, 128, 512, k=0.02)
    caches = (torch.zeros((B, T, cfg.D_I), dtype=torch.bfloat16, device="cuda"),
              torch.zeros((B, T, 576), dtype=torch.bfloat16, device="cuda"))
    kv_len = i32([T])
    ws = dsa.new_workspace(max(dsa.workspace_bytes(op, B, T, T, h, cfg.topk) for op, h in
                               ((dsa.OP_INDEXER_TOPK, cfg.H_I), (dsa.OP_SPARSE_MLA, cfg.H))))
    args = (dsa, cfg, x, residual, gain, W, caches, ws, W_g, W_uv, kv_len)
    s = _layer(*args)
    assert dsa.read_device_status(ws)[0] == dsa.DSA_OK
    # each stage against its 64-bit computation on the stage's own inputs
    d = lambda t: t.double().cpu().numpy()  # noqa: E731
    _check_norm(d(x)[0], d(residual)[0], d(gain), EPS, s["codes"][0], s["scale"][0],
                s["residual"][0], s["y"][0], "layer norm")
    flat = lambda t: t.reshape(B * T, -1)  # noqa: E731
    for name, key in (("q_idx", "q_idx"), ("w", "w"), ("k_pre", "k_pre"), ("kv", "kv_new"),
                      ("q_lat", "q_lat")):
        ref, mag = _linear_ref(flat(s["codes"]), flat(s["scale"]), *W[name])
        _check_linear(flat(s[key]), ref, mag, hid, f"layer {name}")
    rows = np.array([0, 1, 127, 128, 300, 511])
    gi, q_start, kl = s["idx"].cpu().numpy(), np.zeros(1, np.int32), np.array([T], np.int32)
    check_indexer_rows(gi, to_u16(s["q_idx"]), to_u16(s["w"]), to_u16(caches[0]), q_start, kl,
                       cfg.topk, rows, "layer indexer")
    check_mla_rows(to_u16(s["o"]), s["lse"].cpu().numpy(), to_u16(s["q_lat"]), to_u16(caches[1]),
                   gi, q_start, kl, cfg.scale, rows, "layer mla")
    check_gate_rows(to_u16(s["gated"]), to_u16(flat(s["y"])), to_u16(W_g),
                    to_u16(s["o"]).reshape(T, cfg.H, 512), to_u16(W_uv), rows, "layer")
    ref, mag = _linear_ref(s["oc"].view(B * T, -1), s["os"], *W["o"])
    _check_linear(s["out"], ref, mag, cfg.H * 128, "layer output projection")
    # the same layer captured into a graph and replayed on other inputs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = _layer(*args)
    for k in range(2):
        x.copy_(rnd(B, T, hid))
        want = _layer(*args)
        graph.replay()
        torch.cuda.synchronize()
        for n in ("codes", "scale", "residual", "y", "q_idx", "w", "k_pre", "kv_new", "q_lat"):
            assert torch.equal(c[n], want[n]), n
        assert torch.isfinite(c["out"].float()).all()
    assert dsa.read_device_status(ws)[0] == dsa.DSA_OK


# K slices of one block, of fewer blocks than the ring has stages, of as many, of many
# more: the copying and the issuing warp then end in different waits, one lane at a
# time, before the cluster's barriers.
@pytest.mark.parametrize("M,N,K", [(16, 128, 2048), (5, 300, 528), (64, 128, 7168), (40, 1000, 4624),
                                   (3, 129, 12288), (200, 512, 4096), (512, 500, 7168)])
def test_joined_slices_many_times(dsa, M, N, K):
    codes, scale, w_codes, w_scale = _operands(dsa, M + N + K, M, N, K)
    ws = dsa.new_workspace(256)
    out = [torch.empty((M, N), device="cuda") for _ in range(60)]
    for o in out:
        dsa.dsa_linear_fp8(codes, scale, w_codes, w_scale, out=o, workspace=ws)
    assert dsa.read_device_status(ws)[0] == dsa.DSA_OK
    ref, mag = _linear_ref(codes, scale, w_codes, w_scale)
    _check_linear(out[0], ref, mag, K, f"{M}x{N}x{K}")
    assert all(torch.equal(o, out[0]) for o in out)


def test_each_operand_is_refused_by_its_name(dsa):
    """Wrong type, wrong shape, a strided view, another device: for every operand of the
    three calls, the message names it (or says what the shapes have to be together)."""
    codes, scale, w_codes, w_scale = _operands(dsa, 8, 6, 200, 256)
    x, gain = _rows(1, 6, 256), torch.ones(256, dtype=torch.bfloat16, device="cuda")
    calls = [
        (dsa.dsa_rmsnorm_fp8, dict(x=x, gain=gain, residual=x.clone(), codes=torch.empty_like(codes),
                                   scale=torch.empty_like(scale), residual_out=torch.empty_like(x),
                                   y=torch.empty_like(x))),
        (dsa.dsa_quant_fp8_weight, dict(w=x, codes=torch.empty_like(codes),
                                        scale=torch.empty((1, 2), device="cuda"))),
        (dsa.dsa_linear_fp8, dict(codes=codes, scale=scale, w_codes=w_codes, w_scale=w_scale,
                                  out=torch.empty((6, 200), device="cuda"),
                                  workspace=dsa.new_workspace(256)))]
    for call, args in calls:
        call(**args)
        for name, t in args.items():
            strided = torch.zeros((*t.shape, 2), dtype=t.dtype, device="cuda")[..., 0]
            for wrong in (t.to(torch.int16), strided, t.cpu(), [1.0], t.new_zeros((*t.shape, 1))):
                if name == "workspace" and isinstance(wrong, torch.Tensor) and wrong.dim() == 2:
                    continue                                       # any shape will do there
                with pytest.raises((TypeError, ValueError, dsa.DsaError)) as e:
                    call(**dict(args, **{name: wrong}))
                said = str(e.value)
                assert name in said or "must be [" in said, (call.__name__, name, said)
        call(**args)
