"""dsa_rmsnorm_fp8 on rows whose squares FP32 cannot hold: with a small or no eps, values
down to BF16's least.  The checks and bounds are those of test_gpu_linear_fp8: y within
2^-18 (the scaled sum has the same additions, the scaling is by powers of two).  BF16
results may lie outside the range that the oracle rounds in: they are within half a step,
2^-8 of the value, or 2^-134 where they are subnormal."""
import numpy as np
import pytest
import torch

from test_gpu_linear_fp8 import Y_REL, _check_norm, _gen, _rows, dsa  # noqa: F401  (dsa: fixture)

pytestmark = pytest.mark.gpu

# rows share a CTA; one vector per thread; two; four; eight
WIDTHS = [16, 256, 1024, 7168, 16384, 16400, 65536]


def _run(dsa, x, gain, eps, residual=None):
    codes, scale, ro, y = dsa.dsa_rmsnorm_fp8(x, gain, residual=residual, eps=eps, want_y=True)
    return codes, scale, ro, y


def _check(dsa, x, eps, what, residual=None):
    gain = (1 + 0.1 * torch.randn(x.shape[1], generator=_gen(5), device="cuda")).to(torch.bfloat16)
    got = _run(dsa, x, gain, eps, residual)
    d = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    with np.errstate(invalid="ignore"):
        _check_norm(d(x), d(residual), d(gain), eps, got[0], got[1], None, None, what)
    h = d(x) if residual is None else d(x) + d(residual)
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * d(gain)
    for t, want, rel in ((got[2], h, 2.0 ** -24), (got[3], y, Y_REL)):
        if t is not None:
            err, size = np.abs(d(t) - want), np.abs(want)
            assert (err <= (rel + 2.0 ** -8 * (1 + rel)) * size + 2.0 ** -134).all(), what
    return got


@pytest.mark.parametrize("hid", WIDTHS)
@pytest.mark.parametrize("eps", [0.0, 1e-38, 7.8e-31, 8e-31, 1e-20, 1e-5])   # 2^-100 is 7.89e-31
def test_rows_of_every_size(dsa, hid, eps):
    """Rows around 2^-118 to 2^58, ordinary ones among them; with larger eps the small ones
    are made of eps.  7.8e-31 and 8e-31 lie on both sides of 2^-100."""
    x, r = _rows(hid, 12, hid).float(), _rows(hid + 1, 12, hid).float()
    powers = [0., 50., -60., 40., -40., 0., -45., -100., -118., -50., -70., 0.]
    by = torch.exp2(torch.tensor(powers, device="cuda"))[:, None]
    x, r = (x * by).to(torch.bfloat16), (r * by).to(torch.bfloat16)
    assert torch.isfinite(x).all() and (x != 0).any(1).all()
    _check(dsa, x, eps, f"{hid} eps {eps}")
    _check(dsa, x, eps, f"{hid} eps {eps} residual", residual=r)


@pytest.mark.parametrize("hid", [256, 7168])
def test_rows_beside_them_keep_their_bits(dsa, hid):
    gain = torch.ones(hid, dtype=torch.bfloat16, device="cuda")
    x = _rows(hid, 40, hid)
    want = _run(dsa, x, gain, 0.0)
    z = x.clone()
    z[1::3] *= 2.0 ** 100
    z[2::3] *= 2.0 ** -100
    got = _run(dsa, z, gain, 0.0)
    for a, b in zip(want, got):
        if a is not None:
            assert torch.equal(a[::3], b[::3])


def test_subnormal_rows_without_eps(dsa):
    x = torch.full((3, 512), 2.0 ** -133, dtype=torch.bfloat16, device="cuda")
    x[1] = 2.0 ** -126
    x[2] = 0
    gain = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    codes, scale, _, y = _run(dsa, x, gain, 0.0)
    assert (y[:2] == 1).all() and (codes[:2] == 0x7E).all()    # 448
    assert torch.isnan(y[2]).all()                             # 0 / 0
    _, _, _, y = _run(dsa, x, gain, 1e-5)
    assert (y[2] == 0).all()


@pytest.mark.parametrize("eps", [0.0, 1e-5])
def test_a_sum_that_overflows_gives_zeros(dsa, eps):
    x, r = _rows(1, 5, 512), _rows(2, 5, 512)
    x[2] = 2.0 ** 66
    gain = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    codes, _, ro, y = _run(dsa, x, gain, eps, residual=r)
    assert (y[2] == 0).all() and (codes[2] == 0).all() and (ro[2] == 2.0 ** 66).all()
    keep = [0, 1, 3, 4]
    want = _run(dsa, x[keep], gain, eps, residual=r[keep])
    for a, b in zip(want, (codes, None, ro, y)):
        if b is not None:
            assert torch.equal(a, b[keep])
