"""Every kernel of the FP8 projection path by itself, whatever the sizes would have
taken: dsa_linear_fp8's tiles and K slices (by the self-test entry point) with the
forms of storing its output, and the norm's numbers of vectors per thread.  Bounds
and references are those of test_gpu_linear_fp8."""
import ctypes

import pytest
import torch

from linear_kernels import KERNELS
from test_gpu_linear_fp8 import (EPS, _check_linear, _check_norm, _gen, _linear_ref, _operands, _rows,
                                 dsa)  # noqa: F401  (dsa: fixture)

pytestmark = pytest.mark.gpu


def _by(dsa, kernel, codes, scale, w_codes, w_scale, out, ws):
    M, K = codes.shape
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    code = dsa.lib.dsa_selftest_linear_fp8(
        p(codes), p(scale), p(w_codes), p(w_scale), M, w_codes.shape[0], K, p(out),
        0 if out.dtype == torch.bfloat16 else 1, *kernel, p(ws), ws.numel(),
        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert code == dsa.DSA_OK


def _run(dsa, kernel, M, N, K, dtype):
    codes, scale, w_codes, w_scale = _operands(dsa, M + N + K, M, N, K)
    ws = dsa.new_workspace(dsa.workspace_bytes(dsa.OP_LINEAR_FP8, M, 1, K, N, 0))
    buf = torch.full((M * N + 64,), 7.5, dtype=dtype, device="cuda")
    out = buf[:M * N].view(M, N)
    _by(dsa, kernel, codes, scale, w_codes, w_scale, out, ws)
    assert dsa.read_device_status(ws)[0] == dsa.DSA_OK
    ref, mag = _linear_ref(codes, scale, w_codes, w_scale)
    _check_linear(out, ref, mag, K, f"{kernel} {M}x{N}x{K}")
    assert (buf[M * N:] == 7.5).all()
    again = torch.empty_like(out)
    _by(dsa, kernel, codes, scale, w_codes, w_scale, again, ws)
    assert torch.equal(out, again)


# three token tiles, the last of three tokens, and three feature tiles, the last a
# few features wide and stored whole (260) or one by one (261); a block of K for each
# slice (the last of 16 values), and about nine and a half
@pytest.mark.parametrize("tokens,slices", [k for k in KERNELS if k[0] > 0])
@pytest.mark.parametrize("N,dtype", [(260, torch.bfloat16), (261, torch.bfloat16), (260, torch.float32),
                                     (261, torch.float32)])
def test_split_kernel(dsa, tokens, slices, N, dtype):
    M = 2 * tokens + 3
    _run(dsa, (tokens, slices), M, N, 128 * slices - 112, dtype)
    _run(dsa, (tokens, slices), M, N, 128 * (9 * slices + slices // 2 + 1) - 112, dtype)


# a single token and feature; fewer tokens and features than a tile
@pytest.mark.parametrize("tokens,slices", KERNELS)
@pytest.mark.parametrize("M,N", [(1, 1), (7, 100)])
def test_small_calls(dsa, tokens, slices, M, N):
    _run(dsa, (tokens, slices), M, N, 128 * (2 * slices + 1), torch.float32)


# rows of out: by TMA (16-byte boundaries), 4 bytes a lane, 2 bytes a lane; one block
# of K, more than one set of factors; fewer tiles than pairs of SMs and more
@pytest.mark.parametrize("N,dtype", [(520, torch.bfloat16), (518, torch.bfloat16), (517, torch.bfloat16),
                                     (520, torch.float32), (517, torch.float32)])
@pytest.mark.parametrize("M,K", [(3, 16), (259, 128), (259, 4624), (387, 2064), (8200, 144), (8200, 2448)])
def test_wide_kernel(dsa, M, N, K, dtype):
    _run(dsa, (0, 1), M, N, K, dtype)


# the products of a layer's step, in rows that a 64-bit product of all of them is too
# long for: by whatever they take
@pytest.mark.parametrize("M,N,K,dtype", [
    (1, 8192, 7168, torch.bfloat16), (64, 128, 7168, torch.float32), (64, 7168, 12288, torch.bfloat16),
    (2048, 576, 7168, torch.bfloat16), (777, 1001, 1040, torch.float32),
    (16384, 7168, 12288, torch.bfloat16), (64, 55296, 7168, torch.bfloat16),
    (16384, 576, 7168, torch.bfloat16), (75, 3661, 10560, torch.bfloat16),
    (299, 2525, 5472, torch.bfloat16)])
def test_products_of_a_layer(dsa, M, N, K, dtype):
    codes, scale, w_codes, w_scale = _operands(dsa, M + N + K, M, N, K)
    ws = dsa.new_workspace(dsa.workspace_bytes(dsa.OP_LINEAR_FP8, M, 1, K, N, 0))
    out = dsa.dsa_linear_fp8(codes, scale, w_codes, w_scale, out_dtype=dtype, workspace=ws)
    assert dsa.read_device_status(ws)[0] == dsa.DSA_OK
    rows = torch.unique(torch.cat([torch.arange(min(M, 16)), torch.arange(max(0, M - 16), M),
                                   torch.linspace(0, M - 1, 32).long()])).cuda()
    ref, mag = _linear_ref(codes[rows], scale[rows], w_codes, w_scale)
    _check_linear(out[rows], ref, mag, K, f"{M}x{N}x{K}")


# one 16-byte vector per thread, two (of few rows by their width, of many by their
# number), four and eight, at the first and the last width of each
@pytest.mark.parametrize("n,hid", [(2, 1024), (2, 1040), (3, 8192), (3, 8208), (400, 4096), (400, 4112),
                                   (2, 16384), (2, 16400), (2, 32768), (2, 32784), (2, 65536)])
@pytest.mark.parametrize("full", [True, False])
def test_norm_vectors_per_thread(dsa, n, hid, full):
    x = _rows(n + hid, n, hid)
    r = _rows(n + hid + 1, n, hid) if full else None
    gain = (1 + 0.1 * torch.randn(hid, generator=_gen(5), device="cuda")).to(torch.bfloat16)
    codes, scale, ro, y = dsa.dsa_rmsnorm_fp8(x, gain, residual=r, eps=EPS, want_y=full)
    d = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    _check_norm(d(x), d(r), d(gain), EPS, codes, scale, ro, y, f"{n}x{hid}")


def test_large_clusters_in_a_graph(dsa):
    """A product whose K is cut into more than eight slices asks whether their cluster fits;
    captured, with a workspace of the graph's own and with the caller's."""
    codes, scale, w_codes, w_scale = _operands(dsa, 9, 64, 128, 7168)
    ws = dsa.new_workspace(256)
    out = torch.empty((64, 128), device="cuda")
    want = dsa.dsa_linear_fp8(codes, scale, w_codes, w_scale, out=out, workspace=ws).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        own = dsa.dsa_linear_fp8(codes, scale, w_codes, w_scale, out_dtype=torch.float32)
        dsa.dsa_linear_fp8(codes, scale, w_codes, w_scale, out=out, workspace=ws)
    out.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(own, want)
    assert dsa.read_device_status(ws)[0] == dsa.DSA_OK
