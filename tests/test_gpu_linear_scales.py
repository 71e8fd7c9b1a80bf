"""dsa_linear_fp8 with scales whose product leaves FP32's normal range where the output
does not: the quantisers' smallest scale is 2^-109, and FP32 scales may be anything.

Bound: that of test_gpu_linear_fp8 with one more rounded product per block,
(128 + blocks + 3) * 2^-23 of the sum of magnitudes, plus, below FP32's normal range,
half a subnormal step (2^-150) for each block's addition and for the output's rounding;
a BF16 output's subnormal step is 2^-133."""
import pytest
import torch

from test_gpu_linear_fp8 import _linear_ref, _operands, dsa  # noqa: F401  (dsa: fixture)
from test_gpu_linear_kernels import _by

pytestmark = pytest.mark.gpu

# each tile, sliced and not; the wide kernel by TMA (N = 400, both types) and not
SHAPES = [((16, 1), 40, 400), ((16, 4), 40, 400), ((32, 2), 40, 401), ((64, 5), 70, 400),
          ((96, 3), 200, 400), ((128, 2), 200, 401), ((0, 1), 300, 400), ((0, 1), 300, 401)]
K = 2448                      # 20 blocks: more than one set of factors per slice


def _run(dsa, kernel, codes, scale, w_codes, w_scale, dtype):
    ws = dsa.new_workspace(256)
    out = torch.empty((codes.shape[0], w_codes.shape[0]), dtype=dtype, device="cuda")
    _by(dsa, kernel, codes, scale, w_codes, w_scale, out, ws)
    assert dsa.read_device_status(ws)[0] == dsa.DSA_OK
    return out


@pytest.mark.parametrize("kernel,M,N", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_scales_of_any_size(dsa, kernel, M, N, dtype):
    codes, scale, w_codes, w_scale = _operands(dsa, M + N, M, N, K)
    powers = torch.tensor([0., -60., -112., 60., 100.], device="cuda")
    scale = scale * torch.exp2(powers[torch.arange(M, device="cuda") % 5])[:, None]
    w_scale = w_scale * torch.exp2(powers[[2, 0, 1, 4]][:, None])
    # one block of K further off than the others, and one scale below FP32's normal range
    w_scale[1, 7] *= 2.0 ** -50
    scale[0, 3] = 2.0 ** -140
    out = _run(dsa, kernel, codes, scale, w_codes, w_scale, dtype).double()
    ref, mag = _linear_ref(codes, scale, w_codes, w_scale)
    half = torch.finfo(dtype).eps / 2
    kb = -(-K // 128)
    step = 2.0 ** -149 if dtype == torch.float32 else 2.0 ** -133
    tol = (128 + kb + 3) * 2.0 ** -23 * mag * (1 + half) + half * ref.abs() + (kb + 1) * 2.0 ** -150 + step / 2
    fits = mag < 2.0 ** 126                           # no partial sum overflows
    bad = fits & ~((out - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist())
    # the ranges are there: factors that are subnormal or 0 under outputs that are normal
    f = scale.double().amax(1)[:, None] * w_scale.double().amax(1).repeat_interleave(128)[None, :N]
    normal = (f < 2.0 ** -126) & (ref.abs() > 2.0 ** -120)
    assert normal.sum() > 100 and (f > 2.0 ** 128).any()


@pytest.mark.parametrize("kernel,M,N", SHAPES)
def test_factors_beyond_the_largest_number(dsa, kernel, M, N):
    """Products of scales above 2^128: a block's sum of 2^-18 brings them back, one of 0
    gives 0, and an ordinary row beside them keeps its bits."""
    codes, scale, w_codes, w_scale = _operands(dsa, M + N, M, N, K)
    want = _run(dsa, kernel, codes, scale, w_codes, w_scale, torch.float32)
    codes, scale, w_codes, w_scale = (t.clone() for t in (codes, scale, w_codes, w_scale))
    small, zero = 3, 5
    codes[small], codes[zero] = 0, 0
    codes[small, ::128] = 1                           # one code of 2^-9 per block
    scale[small] = 2.0 ** 66
    scale[zero] = 3e38
    w_codes[128:256] = 1
    w_scale[1] = 2.0 ** 64
    w_scale[1, 0] = 3e38
    out = _run(dsa, kernel, codes, scale, w_codes, w_scale, torch.float32)
    blocks = -(-K // 128)
    # 2^-18 * 2^66 * 2^64 for each block but the first, whose 2^-18 * 2^66 * 3e38 overflows
    # for nothing but itself
    assert (out[zero] == 0).all()
    assert torch.isinf(out[small, 128:256]).all()
    w_scale[1, 0] = 2.0 ** 64
    out = _run(dsa, kernel, codes, scale, w_codes, w_scale, torch.float32)
    assert (out[small, 128:256] == blocks * 2.0 ** 112).all()
    rows = [m for m in range(M) if m not in (small, zero)]
    cols = [n for n in range(N) if not 128 <= n < 256]
    assert torch.equal(out[rows][:, cols], want[rows][:, cols])


@pytest.mark.parametrize("kernel,M,N", SHAPES)
def test_products_of_the_quantisers_smallest_scales(dsa, kernel, M, N):
    """Rows of zeros on blocks of zeros, and rows of 2^-99 on weights of 2^-20."""
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[::2] = 2.0 ** -99
    w = torch.full((N, K), 2.0 ** -20, dtype=torch.bfloat16, device="cuda")
    w[:128] = 0
    c, s = dsa.dsa_quant_fp8(torch.nn.functional.pad(x, (0, -K % 128)).view(M, -1, 128).contiguous())
    codes = c.view(M, -1)[:, :K].contiguous()
    w_codes, w_scale = dsa.dsa_quant_fp8_weight(w)
    out = _run(dsa, kernel, codes, s, w_codes, w_scale, torch.float32).double()
    ref, mag = _linear_ref(codes, s, w_codes, w_scale)
    assert (out[1::2] == 0).all() and (out[:, :128] == 0).all()
    kb = -(-K // 128)
    tol = (128 + kb + 3) * 2.0 ** -23 * mag + (kb + 2) * 2.0 ** -150
    assert ((out - ref).abs() <= tol).all() and (out[::2, 128:] > 2.0 ** -120).all()


@pytest.mark.parametrize("kernel,M,N", SHAPES)
def test_non_finite_scales_and_codes_stay_where_they_are(dsa, kernel, M, N):
    """A NaN or an infinite scale, alone, against a scale of 0 and against a subnormal one, and
    NaN codes, beside factors out of range: by the formula, and the others keep their bits."""
    codes, scale, w_codes, w_scale = _operands(dsa, M + N, M, N, K)
    clean = _run(dsa, kernel, codes, scale, w_codes, w_scale, torch.float32)
    codes, scale, w_codes, w_scale = (t.clone() for t in (codes, scale, w_codes, w_scale))
    scale[1, 2] = float("nan")
    scale[2, 9] = float("inf")
    codes[4, 700] = 0x7F                              # a NaN code
    scale[6, 5] = 0.0
    scale[7, 19] = 2.0 ** -149
    w_codes[300, K - 1] = 0xFF
    w_scale[1, 8] = float("nan")
    out = _run(dsa, kernel, codes, scale, w_codes, w_scale, torch.float32)
    nan = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    nan[1] = nan[4] = True
    nan[:, 300] = True
    nan[:, 128:256] = True
    assert torch.isnan(out[nan]).all()
    assert not torch.isfinite(out[2]).any()           # infinite, or infinite times 0
    rest = ~nan
    rest[[2, 6, 7]] = False
    assert torch.equal(out[rest], clean[rest])
    ref, mag = _linear_ref(codes, scale, w_codes, w_scale)
    ok = ~nan
    ok[2] = False
    tol = (128 + -(-K // 128) + 3) * 2.0 ** -23 * mag + 2.0 ** -24 * ref.abs() + 2.0 ** -140
    assert ((out.double() - ref).abs() <= tol)[ok].all()
    # an infinite scale on a scale of 0 is NaN
    scale[2, 9] = 0.0
    w_scale[1, 8] = 1.0
    w_scale[0, 9] = float("inf")
    out = _run(dsa, kernel, codes, scale, w_codes, w_scale, torch.float32)
    assert torch.isnan(out[2, :128]).all() and torch.isfinite(out[2, 128:256]).all()
