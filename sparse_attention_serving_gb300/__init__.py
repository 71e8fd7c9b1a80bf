"""Python binding of libdsa.so, the gated DSA attention step on GB300 (sm_103a).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in ``include/dsa.h``.  PyTorch supplies device
memory and streams.  There is no CPU or PyTorch fallback: importing this
package without a built ``libdsa.so`` raises, and calling an entry point
without a CUDA device fails.

Entry points (same names as the C ABI):
  dsa_indexer_topk  lightning indexer scores + top-k key positions
  sparse_mla_fwd    latent-space attention over the selected rows
  mla_gate_apply    sigmoid output gate applied after the per-head up-projection
  dsa_cache_append  LayerNorm of new indexer keys + append of keys and latent rows
  dsa_quant_fp8, dsa_cache_append_fp8, dsa_indexer_topk_fp8
                    the FP8 (E4M3, one FP32 scale per row) indexer variant
  sparse_mla_bwd    gradients of sparse MLA for q_lat and the latent rows
  dsa_rmsnorm_fp8, dsa_quant_fp8_weight, dsa_linear_fp8
                    the FP8 projections around the step: residual addition + RMS
                    norm to E4M3 codes, a weight's quantisation, the product
  dsa_cache_append_rope
                    dsa_cache_append with positions rotated on the way, in the keys,
                    the latent rows and the queries that go with them
  mla_tree_fwd      dense attention of a tree of drafted tokens over a latent cache
  mla_window_fwd, mla_window_bwd
                    dense attention with a sliding window and first tokens that stay
                    visible, and its gradients
"""

from __future__ import annotations

import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdsa.so")

DSA_OK = 0
DSA_ERR_INVALID_ARGUMENT = 1
DSA_ERR_UNSUPPORTED = 2
DSA_ERR_CUDA = 3
DSA_ERR_DEVICE_TIMEOUT = 4
DSA_ERR_BAD_INDEX = 5
DSA_ERR_WORKSPACE_TOO_SMALL = 6

OP_INDEXER_TOPK, OP_SPARSE_MLA, OP_GATE, OP_CACHE_APPEND, OP_SPARSE_MLA_BWD = 0, 1, 2, 3, 4
OP_LINEAR_FP8 = 5
OP_MLA_TREE, OP_MLA_WINDOW, OP_MLA_WINDOW_BWD = 6, 7, 8
ROPE_NONE, ROPE_HALVES, ROPE_PAIRS = 0, 1, 2   # dims rotated together: (i, i+32) or (2i, 2i+1)
ROPE_DIMS = 64
INDEXER_KEY_EPS = 1e-5   # KimiK3TextConfig rms_norm_eps
RMS_NORM_EPS = 1e-5      # KimiK3TextConfig rms_norm_eps
FP8_BLOCK = 128          # values per scale: along a row, and a weight's rows too
RLAT, VLAT, PAGE = 576, 512, 64
MLA_SCALE = 1.0 / math.sqrt(128 + 64)   # qk_nope_head_dim + qk_rope_head_dim


class DsaError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {status_string(code)} (code {code})")


class _Rows(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("seq_stride", ctypes.c_int64),
                ("block_table", ctypes.c_void_p), ("max_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32)]


EXPORTS = ("dsa_abi_version", "dsa_status_string", "dsa_workspace_bytes", "dsa_workspace_init",
           "dsa_read_device_status", "dsa_indexer_topk", "sparse_mla_fwd", "mla_gate_apply",
           "dsa_cache_append", "sparse_mla_fwd_sink", "dsa_selftest_wait_timeout",
           "dsa_quant_fp8", "dsa_cache_append_fp8", "dsa_indexer_topk_fp8", "sparse_mla_bwd",
           "dsa_rmsnorm_fp8", "dsa_quant_fp8_weight", "dsa_linear_fp8",
           "dsa_selftest_linear_fp8", "dsa_cache_append_rope", "mla_tree_fwd", "mla_window_fwd",
           "mla_window_bwd")


def _load(path: str = LIB_PATH):
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python sparse_attention_serving_gb300/build.py`"
                          " (there is no fallback path)")
    lib = ctypes.CDLL(path)
    P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.dsa_abi_version.restype = I
    lib.dsa_status_string.argtypes = [I]
    lib.dsa_status_string.restype = ctypes.c_char_p
    lib.dsa_workspace_bytes.argtypes = [I, I, I, I, I, I]
    lib.dsa_workspace_bytes.restype = Z
    lib.dsa_workspace_init.argtypes = [P, Z, P]
    lib.dsa_read_device_status.argtypes = [P, P, P, P]
    lib.dsa_indexer_topk.argtypes = [P, P, ctypes.POINTER(_Rows), P, P, I, I, I, I, I, I, P, P, Z, P]
    lib.sparse_mla_fwd.argtypes = [P, ctypes.POINTER(_Rows), P, P, P, I, I, I, I, I,
                                   ctypes.c_float, P, P, P, Z, P]
    lib.sparse_mla_fwd_sink.argtypes = [P, ctypes.POINTER(_Rows), P, P, P, I, I, I, I, I,
                                        ctypes.c_float, P, P, P, P, Z, P]
    lib.mla_gate_apply.argtypes = [P, P, P, P, I, I, I, I, P, P, Z, P]
    lib.dsa_cache_append.argtypes = [P, P, ctypes.POINTER(_Rows), ctypes.POINTER(_Rows), P, I, I, I,
                                     ctypes.c_float, P, Z, P]
    lib.dsa_selftest_wait_timeout.argtypes = [P, Z, ctypes.c_uint64, P]
    lib.dsa_quant_fp8.argtypes = [P, ctypes.c_int64, I, P, P, P]
    lib.dsa_cache_append_fp8.argtypes = [P, P, ctypes.POINTER(_Rows), P, ctypes.POINTER(_Rows), P,
                                         I, I, I, ctypes.c_float, P, Z, P]
    lib.dsa_indexer_topk_fp8.argtypes = [P, P, P, ctypes.POINTER(_Rows), P, P, P, I, I, I, I, I, I,
                                         P, P, Z, P]
    lib.sparse_mla_bwd.argtypes = [P, ctypes.POINTER(_Rows), P, P, P, I, I, I, I, I,
                                   ctypes.c_float, P, P, P, P, P, P, Z, P]
    lib.dsa_rmsnorm_fp8.argtypes = [P, P, P, ctypes.c_int64, I, ctypes.c_float, P, P, P, P, P]
    lib.dsa_quant_fp8_weight.argtypes = [P, I, I, P, P, P]
    lib.dsa_linear_fp8.argtypes = [P, P, P, P, I, I, I, P, I, P, Z, P]
    lib.dsa_selftest_linear_fp8.argtypes = [P, P, P, P, I, I, I, P, I, I, I, P, Z, P]
    rows = ctypes.POINTER(_Rows)
    lib.dsa_cache_append_rope.argtypes = [P, P, rows, rows, P, P, I, P, P, P, P, I, P, P, I, I, I, I,
                                          I, I, ctypes.c_float, P, Z, P]
    lib.mla_tree_fwd.argtypes = [P, rows, P, P, P, I, I, I, I, ctypes.c_float, P, P, P, Z, P]
    lib.mla_window_fwd.argtypes = [P, rows, P, P, I, I, I, I, I, I, ctypes.c_float, P, P, P, Z, P]
    lib.mla_window_bwd.argtypes = [P, rows, P, P, I, I, I, I, I, I, ctypes.c_float, P, P, P, P, P,
                                   P, Z, P]
    for f in ("dsa_cache_append_rope", "mla_tree_fwd", "mla_window_fwd", "mla_window_bwd",
              "dsa_selftest_linear_fp8", "dsa_rmsnorm_fp8", "dsa_quant_fp8_weight", "dsa_linear_fp8",
              "sparse_mla_bwd", "dsa_workspace_init", "dsa_read_device_status", "dsa_indexer_topk",
              "sparse_mla_fwd", "mla_gate_apply", "dsa_cache_append", "sparse_mla_fwd_sink",
              "dsa_selftest_wait_timeout", "dsa_quant_fp8", "dsa_cache_append_fp8",
              "dsa_indexer_topk_fp8"):
        getattr(lib, f).restype = I
    return lib


lib = _load()


def status_string(code: int) -> str:
    return lib.dsa_status_string(int(code)).decode()


def _check(code: int, what: str):
    if code != DSA_OK:
        raise DsaError(code, what)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _need(t: torch.Tensor, dtype, name: str):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise DsaError(DSA_ERR_INVALID_ARGUMENT, f"{name} must be on a CUDA device")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise DsaError(DSA_ERR_INVALID_ARGUMENT, f"{name} must be contiguous")


class Rows:
    """A per-token row store: contiguous ``[B, S, width]`` or a paged pool
    ``[num_pages, 64, width]`` with ``block_table [B, max_pages]`` (int32).
    BF16 rows, or uint8 rows of E4M3 codes for the FP8 indexer variant."""

    def __init__(self, base: torch.Tensor, block_table: torch.Tensor | None = None,
                 seq_stride: int | None = None):
        _need(base, torch.uint8 if base.dtype == torch.uint8 else torch.bfloat16, "rows.base")
        self.base = base
        self.block_table = block_table
        if block_table is None:
            if base.dim() != 3:
                raise ValueError("contiguous rows must be [B, S, width]")
            self.seq_stride = base.shape[1] if seq_stride is None else seq_stride
            self.num_pages = 0
            self.max_pages = 0
        else:
            _need(block_table, torch.int32, "block_table")
            if base.dim() != 3 or base.shape[1] != PAGE:
                raise ValueError("paged rows must be [num_pages, 64, width]")
            self.seq_stride = 0
            self.num_pages = base.shape[0]
            self.max_pages = block_table.shape[1]
        self._key = self._pointer = None

    def _p(self):
        """A pointer to the C struct, made anew when a field has changed (the struct and its
        pointer take 1.5 us)."""
        table = self.block_table
        key = (self.base.data_ptr(), table is not None and table.data_ptr(), self.seq_stride,
               self.max_pages, self.num_pages)
        if key != self._key:
            self._pointer, self._key = ctypes.pointer(self.c()), key
        return self._pointer

    def c(self) -> _Rows:
        table = self.block_table
        if table is None:
            return _Rows(self.base.data_ptr(), int(self.seq_stride), 0, int(self.max_pages), 0,
                         int(self.num_pages))
        return _Rows(self.base.data_ptr(), int(self.seq_stride), table.data_ptr(), int(self.max_pages),
                     PAGE, int(self.num_pages))


def workspace_bytes(op: int, B: int, Tq: int, max_kv_len: int, heads: int, topk: int) -> int:
    return int(lib.dsa_workspace_bytes(op, B, Tq, max_kv_len, heads, topk))


def new_workspace(nbytes: int, device=None, stream=None) -> torch.Tensor:
    """Allocate (through torch) and initialise a workspace of at least nbytes."""
    nbytes = max(256, (int(nbytes) + 255) // 256 * 256)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")
    _check(lib.dsa_workspace_init(_ptr(ws), nbytes, _stream(stream)), "dsa_workspace_init")
    return ws


def read_device_status(workspace: torch.Tensor, stream=None):
    """Synchronise the stream, return (code, where, detail) and clear the status."""
    where, detail = ctypes.c_uint32(0), ctypes.c_uint32(0)
    code = lib.dsa_read_device_status(_ptr(workspace), _stream(stream), ctypes.byref(where),
                                      ctypes.byref(detail))
    return int(code), int(where.value), int(detail.value)


def selftest_wait_timeout(workspace: torch.Tensor, limit_ns: int = 20_000_000, stream=None):
    """Run the device failure-path self-test; returns (code, where, detail) read back."""
    _check(lib.dsa_selftest_wait_timeout(_ptr(workspace), workspace.numel(), int(limit_ns),
                                         _stream(stream)), "dsa_selftest_wait_timeout")
    return read_device_status(workspace, stream)


def _ws(workspace, op, B, Tq, max_kv_len, heads, topk, device, stream):
    need = workspace_bytes(op, B, Tq, max_kv_len, heads, topk)
    if workspace is None:
        workspace = new_workspace(need, device, stream)
    _need(workspace, torch.uint8, "workspace")
    return workspace


def dsa_indexer_topk(q_idx, w, k_idx: Rows, q_start, kv_len, topk: int, max_kv_len: int,
                     out_idx=None, workspace=None, stream=None):
    """q_idx [B,Tq,H_I,D_I] bf16, w [B,Tq,H_I] bf16, k_idx Rows (width D_I),
    q_start/kv_len [B] int32 -> out_idx [B,Tq,topk] int32 (-1 padded)."""
    _need(q_idx, torch.bfloat16, "q_idx")
    _need(w, torch.bfloat16, "w")
    _need(q_start, torch.int32, "q_start")
    _need(kv_len, torch.int32, "kv_len")
    B, Tq, H_I, D_I = q_idx.shape
    if out_idx is None:
        out_idx = torch.empty((B, Tq, topk), dtype=torch.int32, device=q_idx.device)
    _need(out_idx, torch.int32, "out_idx")
    ws = _ws(workspace, OP_INDEXER_TOPK, B, Tq, max_kv_len, H_I, topk, q_idx.device, stream)
    rows = k_idx.c()
    _check(lib.dsa_indexer_topk(_ptr(q_idx), _ptr(w), ctypes.byref(rows), _ptr(q_start),
                                _ptr(kv_len), B, Tq, H_I, D_I, int(max_kv_len), int(topk),
                                _ptr(out_idx), _ptr(ws), ws.numel(), _stream(stream)),
           "dsa_indexer_topk")
    return out_idx


def sparse_mla_fwd(q_lat, kv: Rows, idx, q_start, kv_len, max_kv_len: int, scale: float = MLA_SCALE,
                   o_lat=None, lse=None, want_lse: bool = True, workspace=None, stream=None,
                   sink=None):
    """q_lat [B,Tq,H,576] bf16, kv Rows (width 576), idx [B,Tq,topk] int32 ->
    (o_lat [B,Tq,H,512] bf16, lse [B,Tq,H] float32 or None).  sink: optional [H]
    float32 learnable sink logits (calls sparse_mla_fwd_sink)."""
    _need(q_lat, torch.bfloat16, "q_lat")
    _need(idx, torch.int32, "idx")
    _need(q_start, torch.int32, "q_start")
    _need(kv_len, torch.int32, "kv_len")
    B, Tq, H, R = q_lat.shape
    topk = idx.shape[-1]
    if o_lat is None:
        o_lat = torch.empty((B, Tq, H, VLAT), dtype=torch.bfloat16, device=q_lat.device)
    _need(o_lat, torch.bfloat16, "o_lat")
    if lse is None and want_lse:
        lse = torch.empty((B, Tq, H), dtype=torch.float32, device=q_lat.device)
    if lse is not None:
        _need(lse, torch.float32, "lse")
    ws = _ws(workspace, OP_SPARSE_MLA, B, Tq, max_kv_len, H, topk, q_lat.device, stream)
    rows = kv.c()
    if sink is None:
        _check(lib.sparse_mla_fwd(_ptr(q_lat), ctypes.byref(rows), _ptr(idx), _ptr(q_start),
                                  _ptr(kv_len), B, Tq, H, topk, int(max_kv_len), float(scale),
                                  _ptr(o_lat), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)),
               "sparse_mla_fwd")
    else:
        _need(sink, torch.float32, "sink")
        if tuple(sink.shape) != (H,):
            raise ValueError("sink must be [H]")
        _check(lib.sparse_mla_fwd_sink(_ptr(q_lat), ctypes.byref(rows), _ptr(idx), _ptr(q_start),
                                       _ptr(kv_len), B, Tq, H, topk, int(max_kv_len),
                                       float(scale), _ptr(sink), _ptr(o_lat), _ptr(lse),
                                       _ptr(ws), ws.numel(), _stream(stream)),
               "sparse_mla_fwd_sink")
    return o_lat, lse


def mla_gate_apply(x, W_g, o_lat, W_uv, out=None, workspace=None, stream=None):
    """x [N,hid] bf16, W_g [H*dv,hid] bf16, o_lat [N,H,512] bf16, W_uv [H,dv,512] bf16
    -> out [N, H*dv] bf16."""
    for t, n in ((x, "x"), (W_g, "W_g"), (o_lat, "o_lat"), (W_uv, "W_uv")):
        _need(t, torch.bfloat16, n)
    N, hid = x.shape
    H, dv, R = W_uv.shape
    if out is None:
        out = torch.empty((N, H * dv), dtype=torch.bfloat16, device=x.device)
    _need(out, torch.bfloat16, "out")
    ws = _ws(workspace, OP_GATE, N, 1, 0, H, 0, x.device, stream)
    _check(lib.mla_gate_apply(_ptr(x), _ptr(W_g), _ptr(o_lat), _ptr(W_uv), N, hid, H, dv,
                              _ptr(out), _ptr(ws), ws.numel(), _stream(stream)),
           "mla_gate_apply")
    return out


def dsa_cache_append(k_pre, kv_new, k_cache: Rows, kv_cache: Rows, q_start,
                     eps: float = INDEXER_KEY_EPS, workspace=None, stream=None):
    """k_pre [B,Tq,D_I] float32, kv_new [B,Tq,576] bf16, caches as Rows (written in
    place), q_start [B] int32: LayerNorm'd BF16 keys and the latent rows land at
    positions q_start[b]+i.  Returns the workspace (its status word holds any
    BAD_INDEX raised for rows the caches do not have)."""
    _need(k_pre, torch.float32, "k_pre")
    _need(kv_new, torch.bfloat16, "kv_new")
    _need(q_start, torch.int32, "q_start")
    B, Tq, D_I = k_pre.shape
    if tuple(kv_new.shape) != (B, Tq, RLAT):
        raise ValueError("kv_new must be [B, Tq, 576]")
    ws = _ws(workspace, OP_CACHE_APPEND, B, Tq, 0, 0, 0, k_pre.device, stream)
    kr, vr = k_cache.c(), kv_cache.c()
    _check(lib.dsa_cache_append(_ptr(k_pre), _ptr(kv_new), ctypes.byref(kr), ctypes.byref(vr),
                                _ptr(q_start), B, Tq, D_I, float(eps), _ptr(ws), ws.numel(),
                                _stream(stream)), "dsa_cache_append")
    return ws


# ---------------------------------------------------------------------------
# FP8 (E4M3) indexer variant
# ---------------------------------------------------------------------------

def dsa_quant_fp8(x, codes=None, scale=None, stream=None):
    """x [..., D] bf16 (D in {64, 128}) -> (codes [..., D] uint8, scale [...] float32):
    scale = max(amax, 2^-100)/448 per row, code = E4M3(x * (1/scale))."""
    _need(x, torch.bfloat16, "x")
    D = x.shape[-1]
    n = x.numel() // D if D else 0
    if codes is None:
        codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    if scale is None:
        scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    _need(codes, torch.uint8, "codes")
    _need(scale, torch.float32, "scale")
    _check(lib.dsa_quant_fp8(_ptr(x), n, D, _ptr(codes), _ptr(scale), _stream(stream)),
           "dsa_quant_fp8")
    return codes, scale


def dsa_cache_append_fp8(k_pre, kv_new, k_codes: Rows, k_scale, kv_cache: Rows, q_start,
                         eps: float = INDEXER_KEY_EPS, workspace=None, stream=None):
    """dsa_cache_append with the key stored as E4M3 codes (k_codes, uint8 rows of
    D_I) plus one float32 scale per row (k_scale, laid out like k_codes' rows:
    [B, S] contiguous or [num_pages, 64] paged).  Returns the workspace."""
    _need(k_pre, torch.float32, "k_pre")
    _need(kv_new, torch.bfloat16, "kv_new")
    _need(q_start, torch.int32, "q_start")
    _need(k_scale, torch.float32, "k_scale")
    B, Tq, D_I = k_pre.shape
    if tuple(kv_new.shape) != (B, Tq, RLAT):
        raise ValueError("kv_new must be [B, Tq, 576]")
    ws = _ws(workspace, OP_CACHE_APPEND, B, Tq, 0, 0, 0, k_pre.device, stream)
    kr, vr = k_codes.c(), kv_cache.c()
    _check(lib.dsa_cache_append_fp8(_ptr(k_pre), _ptr(kv_new), ctypes.byref(kr), _ptr(k_scale),
                                    ctypes.byref(vr), _ptr(q_start), B, Tq, D_I, float(eps),
                                    _ptr(ws), ws.numel(), _stream(stream)),
           "dsa_cache_append_fp8")
    return ws


def dsa_indexer_topk_fp8(q_codes, q_scale, w, k_codes: Rows, k_scale, q_start, kv_len, topk: int,
                         max_kv_len: int, out_idx=None, workspace=None, stream=None):
    """q_codes [B,Tq,H_I,D_I] uint8, q_scale [B,Tq,H_I] float32, w [B,Tq,H_I] bf16,
    k_codes Rows (uint8, width D_I), k_scale float32 laid out like k_codes' rows
    -> out_idx [B,Tq,topk] int32 (-1 padded)."""
    _need(q_codes, torch.uint8, "q_codes")
    _need(q_scale, torch.float32, "q_scale")
    _need(w, torch.bfloat16, "w")
    _need(k_scale, torch.float32, "k_scale")
    _need(q_start, torch.int32, "q_start")
    _need(kv_len, torch.int32, "kv_len")
    B, Tq, H_I, D_I = q_codes.shape
    if out_idx is None:
        out_idx = torch.empty((B, Tq, topk), dtype=torch.int32, device=q_codes.device)
    _need(out_idx, torch.int32, "out_idx")
    ws = _ws(workspace, OP_INDEXER_TOPK, B, Tq, max_kv_len, H_I, topk, q_codes.device, stream)
    rows = k_codes.c()
    _check(lib.dsa_indexer_topk_fp8(_ptr(q_codes), _ptr(q_scale), _ptr(w), ctypes.byref(rows),
                                    _ptr(k_scale), _ptr(q_start), _ptr(kv_len), B, Tq, H_I, D_I,
                                    int(max_kv_len), int(topk), _ptr(out_idx), _ptr(ws),
                                    ws.numel(), _stream(stream)), "dsa_indexer_topk_fp8")
    return out_idx


def sparse_mla_bwd(q_lat, kv: Rows, idx, q_start, kv_len, max_kv_len: int, o_lat, lse, d_o,
                   dkv, scale: float = MLA_SCALE, dq=None, workspace=None, stream=None):
    """Backward of sparse_mla_fwd for a fixed index set: returns dq [B,Tq,H,576]
    float32 and ADDS the latent-row gradients into dkv (float32, laid out like
    kv's rows: [B, S, 576] or [num_pages, 64, 576]; zero it first)."""
    _need(q_lat, torch.bfloat16, "q_lat")
    _need(idx, torch.int32, "idx")
    _need(o_lat, torch.bfloat16, "o_lat")
    _need(lse, torch.float32, "lse")
    _need(d_o, torch.bfloat16, "d_o")
    _need(dkv, torch.float32, "dkv")
    _need(q_start, torch.int32, "q_start")
    _need(kv_len, torch.int32, "kv_len")
    B, Tq, H, _ = q_lat.shape
    topk = idx.shape[-1]
    if dq is None:
        dq = torch.empty((B, Tq, H, RLAT), dtype=torch.float32, device=q_lat.device)
    _need(dq, torch.float32, "dq")
    ws = _ws(workspace, OP_SPARSE_MLA_BWD, B, Tq, 0, 0, 0, q_lat.device, stream)
    rows = kv.c()
    _check(lib.sparse_mla_bwd(_ptr(q_lat), ctypes.byref(rows), _ptr(idx), _ptr(q_start),
                              _ptr(kv_len), B, Tq, H, topk, int(max_kv_len), float(scale),
                              _ptr(o_lat), _ptr(lse), _ptr(d_o), _ptr(dq), _ptr(dkv), _ptr(ws),
                              ws.numel(), _stream(stream)), "sparse_mla_bwd")
    return dq


# ---------------------------------------------------------------------------
# FP8 projections around the step
# ---------------------------------------------------------------------------

def _refuse(call: str, dev: int, *operands):
    """Refuse a call whose operands, each (tensor, types, shape, name), are not all of one
    of their types (None: any), of their shape (None: any), contiguous and on the device:
    by the first that is not.  Never returns: the calls check all of it in one expression
    first (1 us less of a call's 9), and one that fails there is refused whatever is found."""
    for t, dtypes, shape, name in operands:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype not in dtypes:
            raise TypeError(f"{name} must be {' or '.join(str(d)[6:] for d in dtypes)}, got {t.dtype}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
        if not t.is_contiguous():
            raise DsaError(DSA_ERR_INVALID_ARGUMENT, f"{name} must be contiguous")
        if t.get_device() != dev:
            raise DsaError(DSA_ERR_INVALID_ARGUMENT, f"{name} must be on cuda:{dev}")
    raise DsaError(DSA_ERR_INVALID_ARGUMENT, f"{call}: operands")


def _device(t, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dev = t.get_device()
    if dev < 0:
        raise DsaError(DSA_ERR_INVALID_ARGUMENT, f"{name} must be on a CUDA device")
    return dev


# The current stream's handle and the current device without building objects,
# where torch has them: a call's host time is most of a small call's time.
_current_raw = getattr(torch._C, "_cuda_getCurrentRawStream",
                       lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_on(dev: int, stream) -> int:
    if stream is None:
        return _current_raw(dev)
    if stream.device_index != dev:
        raise DsaError(DSA_ERR_INVALID_ARGUMENT, f"stream must be on cuda:{dev}")
    return stream.cuda_stream


def _empty(shape, dtype, dev: int, stream):
    """An output that belongs to the launch stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


_BF16, _U8, _F32 = torch.bfloat16, torch.uint8, torch.float32
_SIZES = 1 << 30   # sizes at and beyond it are refused here: the C ABI's are 32-bit


def _too_large(call: str, **sizes):
    got = ", ".join(f"{n} = {v}" for n, v in sizes.items())
    raise DsaError(DSA_ERR_UNSUPPORTED, f"{call}: {got}, all below 2^30")


def dsa_rmsnorm_fp8(x, gain, residual=None, eps: float = RMS_NORM_EPS, codes=None, scale=None,
                    residual_out=None, y=None, want_y: bool = False, stream=None):
    """x [..., hid] bf16, gain [hid] bf16, residual like x or None ->
    (codes [..., hid] uint8, scale [..., ceil(hid/128)] float32, residual_out, y):
    h = x + residual, v = h / sqrt(mean(h^2) + eps) * gain, codes and scales the
    E4M3 groups of 128 of v, residual_out = bf16(h) (None without a residual) and
    y = bf16(v) (None unless y is given or want_y).  residual_out and y may be x
    or residual themselves."""
    dev = _device(x, "x")
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return dsa_rmsnorm_fp8(x, gain, residual, eps, codes, scale, residual_out, y, want_y,
                                   stream)
    raw = _stream_on(dev, stream)
    shape = x.shape
    if not shape:
        raise ValueError("x must be [..., hid]")
    hid = shape[-1]
    if hid >= _SIZES:
        _too_large("dsa_rmsnorm_fp8", hid=hid)
    groups = (*shape[:-1], -(-hid // FP8_BLOCK))
    if codes is None:
        codes = _empty(shape, _U8, dev, stream)
    if scale is None:
        scale = _empty(groups, _F32, dev, stream)
    if residual is not None and residual_out is None:
        residual_out = _empty(shape, _BF16, dev, stream)
    if y is None and want_y:
        y = _empty(shape, _BF16, dev, stream)
    try:
        good = (x.dtype is _BF16 and gain.dtype is _BF16 and codes.dtype is _U8
                and scale.dtype is _F32 and gain.shape == (hid,) and codes.shape == shape
                and scale.shape == groups and x.is_contiguous() and gain.is_contiguous()
                and codes.is_contiguous() and scale.is_contiguous()
                and dev == gain.get_device() == codes.get_device() == scale.get_device())
        for t in (residual, residual_out, y):
            if t is not None:
                good = (good and t.dtype is _BF16 and t.shape == shape and t.is_contiguous()
                        and t.get_device() == dev)
    except AttributeError:
        good = False
    if not good:
        _refuse("dsa_rmsnorm_fp8", dev, (x, (_BF16,), None, "x"), (gain, (_BF16,), (hid,), "gain"),
                (codes, (_U8,), shape, "codes"), (scale, (_F32,), groups, "scale"),
                *((t, (_BF16,), shape, name) for t, name in
                  ((residual, "residual"), (residual_out, "residual_out"), (y, "y")) if t is not None))
    code = lib.dsa_rmsnorm_fp8(
        x.data_ptr(), None if residual is None else residual.data_ptr(), gain.data_ptr(),
        x.numel() // hid if hid else 0, hid, eps,
        None if residual_out is None else residual_out.data_ptr(),
        None if y is None else y.data_ptr(), codes.data_ptr(), scale.data_ptr(), raw)
    if code:
        raise DsaError(code, "dsa_rmsnorm_fp8")
    return codes, scale, residual_out, y


def dsa_quant_fp8_weight(w, codes=None, scale=None, stream=None):
    """w [N,K] bf16 (one row per output feature) -> (codes [N,K] uint8,
    scale [ceil(N/128), ceil(K/128)] float32), one scale per 128 x 128 block."""
    dev = _device(w, "w")
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return dsa_quant_fp8_weight(w, codes, scale, stream)
    raw = _stream_on(dev, stream)
    shape = w.shape
    if len(shape) != 2:
        raise ValueError("w must be [N, K]")
    N, K = shape
    if N >= _SIZES or K >= _SIZES:
        _too_large("dsa_quant_fp8_weight", N=N, K=K)
    groups = (-(-N // FP8_BLOCK), -(-K // FP8_BLOCK))
    if codes is None:
        codes = _empty(shape, _U8, dev, stream)
    if scale is None:
        scale = _empty(groups, _F32, dev, stream)
    try:
        good = (w.dtype is _BF16 and codes.dtype is _U8 and scale.dtype is _F32
                and codes.shape == shape and scale.shape == groups and w.is_contiguous()
                and codes.is_contiguous() and scale.is_contiguous()
                and dev == codes.get_device() == scale.get_device())
    except AttributeError:
        good = False
    if not good:
        _refuse("dsa_quant_fp8_weight", dev, (w, (_BF16,), None, "w"),
                (codes, (_U8,), shape, "codes"), (scale, (_F32,), groups, "scale"))
    code = lib.dsa_quant_fp8_weight(w.data_ptr(), N, K, codes.data_ptr(), scale.data_ptr(), raw)
    if code:
        raise DsaError(code, "dsa_quant_fp8_weight")
    return codes, scale


_DTYPES = {torch.bfloat16: 0, torch.float32: 1}   # dsa_dtype_t


def dsa_linear_fp8(codes, scale, w_codes, w_scale, out=None, out_dtype=torch.bfloat16,
                   workspace=None, stream=None):
    """codes [..., K] uint8 with scale [..., ceil(K/128)] float32 (dsa_rmsnorm_fp8, or
    dsa_quant_fp8 of rows of 128), w_codes [N,K] uint8 with w_scale
    [ceil(N/128), ceil(K/128)] float32 (dsa_quant_fp8_weight) -> out [..., N] of
    out_dtype (bfloat16 or float32; out's own when it is given)."""
    dev = _device(codes, "codes")
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return dsa_linear_fp8(codes, scale, w_codes, w_scale, out, out_dtype, workspace, stream)
    raw = _stream_on(dev, stream)
    if not isinstance(w_codes, torch.Tensor):
        raise TypeError("w_codes must be a torch.Tensor")
    shape, w_shape = codes.shape, w_codes.shape
    if len(w_shape) != 2 or not shape or shape[-1] != w_shape[1]:
        raise ValueError("codes must be [..., K] and w_codes [N, K]")
    N, K = w_shape
    M = codes.numel() // K if K else 0
    if M >= _SIZES or N >= _SIZES or K >= _SIZES:
        _too_large("dsa_linear_fp8", M=M, N=N, K=K)
    kb = -(-K // FP8_BLOCK)
    lead = shape[:-1]
    out_shape = (*lead, N)
    w_groups = (-(-N // FP8_BLOCK), kb)
    if out is None:
        if out_dtype not in _DTYPES:
            raise TypeError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
        out = _empty(out_shape, out_dtype, dev, stream)
    if workspace is None:
        need = workspace_bytes(OP_LINEAR_FP8, M, 1, K, N, 0)
        workspace = _empty((need,), _U8, dev, stream)
        _check(lib.dsa_workspace_init(workspace.data_ptr(), need, raw), "dsa_workspace_init")
    try:
        good = (codes.dtype is _U8 and w_codes.dtype is _U8 and scale.dtype is _F32
                and w_scale.dtype is _F32 and out.dtype in _DTYPES and workspace.dtype is _U8
                and scale.shape == (*lead, kb) and w_scale.shape == w_groups
                and out.shape == out_shape and codes.is_contiguous() and w_codes.is_contiguous()
                and scale.is_contiguous() and w_scale.is_contiguous() and out.is_contiguous()
                and workspace.is_contiguous()
                and dev == w_codes.get_device() == scale.get_device() == w_scale.get_device()
                == out.get_device() == workspace.get_device())
    except AttributeError:
        good = False
    if not good:
        _refuse("dsa_linear_fp8", dev, (codes, (_U8,), None, "codes"),
                (scale, (_F32,), (*lead, kb), "scale"), (w_codes, (_U8,), None, "w_codes"),
                (w_scale, (_F32,), w_groups, "w_scale"), (out, tuple(_DTYPES), out_shape, "out"),
                (workspace, (_U8,), None, "workspace"))
    code = lib.dsa_linear_fp8(codes.data_ptr(), scale.data_ptr(), w_codes.data_ptr(),
                              w_scale.data_ptr(), M, N, K, out.data_ptr(), _DTYPES[out.dtype],
                              workspace.data_ptr(), workspace.numel(), raw)
    if code:
        raise DsaError(code, "dsa_linear_fp8")
    return out


# ---------------------------------------------------------------------------
# Rotated positions, and dense attention over latent rows
# ---------------------------------------------------------------------------

_I32, _I64 = torch.int32, torch.int64
_INT = 1 << 31


def _rows_good(rows, B: int, width: int, need_rows: int, dev: int) -> bool:
    """Whether a row store holds BF16 rows of `width`, at least `need_rows` of each of B
    sequences, on the device."""
    base, table = rows.base, rows.block_table
    shape = base.shape
    return (base.dtype is _BF16 and shape[2] == width and base.get_device() == dev
            and ((B - 1) * rows.seq_stride + need_rows <= shape[0] * shape[1] if table is None else
                 len(table.shape) == 2 and table.shape[0] >= B and table.get_device() == dev))


def _refuse_rows(rows, B: int, width: int, need_rows: int, dev: int, name: str):
    """Refuse a row store that _rows_good does not accept, by what is wrong with it."""
    if not isinstance(rows, Rows):
        raise TypeError(f"{name} must be Rows")
    base, table = rows.base, rows.block_table
    if base.dtype is not _BF16:
        raise TypeError(f"{name} must hold bfloat16 rows, got {base.dtype}")
    if base.shape[2] != width:
        raise ValueError(f"{name} must hold rows of {width}, got {base.shape[2]}")
    if base.get_device() != dev or (table is not None and table.get_device() != dev):
        raise DsaError(DSA_ERR_INVALID_ARGUMENT, f"{name} must be on cuda:{dev}")
    if table is not None:
        if table.dim() != 2 or table.shape[0] < B:
            raise ValueError(f"{name}'s block_table must be [B, max_pages]")
    elif (B - 1) * rows.seq_stride + need_rows > base.shape[0] * base.shape[1]:
        raise ValueError(f"{name} has fewer rows than {B} sequences of {need_rows} every "
                         f"{rows.seq_stride}")


def _queries(call: str, q_lat):
    """B, T, H of q_lat [B, T, H, 576]."""
    shape = q_lat.shape
    if len(shape) != 4 or shape[3] != RLAT:
        raise ValueError(f"q_lat must be [B, T, H, {RLAT}], got {list(shape)}")
    B, T, H, _ = shape
    if B >= _SIZES or T >= _SIZES or H >= _SIZES:
        _too_large(call, B=B, T=T, H=H)
    return B, T, H


def _ints(call: str, **sizes):
    for name, v in sizes.items():
        if not isinstance(v, int):
            raise TypeError(f"{name} must be an int")
        if not -_INT <= v < _INT:
            raise DsaError(DSA_ERR_UNSUPPORTED, f"{call}: {name} = {v}")


def _workspace_for(dev: int, stream, raw: int, *sizes):
    need = workspace_bytes(*sizes)
    workspace = _empty((need,), _U8, dev, stream)
    _check(lib.dsa_workspace_init(workspace.data_ptr(), need, raw), "dsa_workspace_init")
    return workspace


def _zeros(shape, dtype, dev: int, stream):
    if stream is None:
        return torch.zeros(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.zeros(shape, dtype=dtype, device=dev)


def _at(t):
    return None if t is None else t.data_ptr()


def _all_good(dev: int, *operands) -> bool:
    """Whether every operand (tensor or None, type, shape) is of its type and shape,
    contiguous and on the device."""
    for t, dtype, shape in operands:
        if t is not None and not (t.dtype is dtype and t.shape == shape and t.is_contiguous()
                                  and t.get_device() == dev):
            return False
    return True


def dsa_cache_append_rope(k_pre, kv_new, k_cache: Rows, kv_cache: Rows, q_start, rope, pos=None,
                          n_new=None, q_pe=None, q_lat=None, q_idx=None, q_idx_out=None,
                          kv_style: int = ROPE_HALVES, key_style: int = ROPE_HALVES,
                          eps: float = INDEXER_KEY_EPS, workspace=None, stream=None):
    """dsa_cache_append with rotated positions.  k_pre [B,Tq,D_I] float32, kv_new [B,Tq,576]
    bf16, caches as Rows (written in place), q_start [B] int32, rope [n_pos,64] float32 (32
    cosines, 32 sines per position), pos [B,Tq] int32 (None: q_start[b]+i), n_new [B] int32
    tokens that are there (None: Tq).  q_pe [B,Tq,H,64] bf16 is rotated into dims 512..575 of
    q_lat [B,Tq,H,576] bf16; q_idx [B,Tq,H_I,D_I] bf16 into q_idx_out (None: in place).
    Returns the workspace (its status word holds any BAD_INDEX)."""
    dev = _device(k_pre, "k_pre")
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return dsa_cache_append_rope(k_pre, kv_new, k_cache, kv_cache, q_start, rope, pos, n_new,
                                         q_pe, q_lat, q_idx, q_idx_out, kv_style, key_style, eps,
                                         workspace, stream)
    raw = _stream_on(dev, stream)
    shape = k_pre.shape
    if len(shape) != 3:
        raise ValueError("k_pre must be [B, Tq, D_I]")
    B, Tq, D_I = shape
    if B >= _SIZES or Tq >= _SIZES or D_I >= _SIZES:
        _too_large("dsa_cache_append_rope", B=B, Tq=Tq, D_I=D_I)
    if (q_pe is None) != (q_lat is None):
        raise ValueError("q_pe and q_lat go together")
    if q_idx is None and q_idx_out is not None:
        raise ValueError("q_idx_out needs q_idx")
    if q_idx_out is None:
        q_idx_out = q_idx
    for t, name in ((rope, "rope"), (q_pe, "q_pe"), (q_idx, "q_idx")):
        if not isinstance(t, torch.Tensor) and (t is not None or name == "rope"):
            raise TypeError(f"{name} must be a torch.Tensor")
    n_pos = rope.shape[0] if rope.shape else 0
    H = 0 if q_pe is None else q_pe.shape[2] if len(q_pe.shape) == 4 else 0
    H_I = 0 if q_idx is None else q_idx.shape[2] if len(q_idx.shape) == 4 else 0
    if n_pos >= _SIZES or H >= _SIZES or H_I >= _SIZES:
        _too_large("dsa_cache_append_rope", n_pos=n_pos, H=H, H_I=H_I)
    if workspace is None:
        workspace = _workspace_for(dev, stream, raw, OP_CACHE_APPEND, B, Tq, 0, 0, 0)
    try:
        good = (_all_good(dev, (k_pre, _F32, shape), (kv_new, _BF16, (B, Tq, RLAT)),
                          (q_start, _I32, (B,)), (rope, _F32, (n_pos, ROPE_DIMS)),
                          (pos, _I32, (B, Tq)), (n_new, _I32, (B,)),
                          (q_pe, _BF16, (B, Tq, H, ROPE_DIMS)), (q_lat, _BF16, (B, Tq, H, RLAT)),
                          (q_idx, _BF16, (B, Tq, H_I, D_I)))
                and (q_idx_out is q_idx or _all_good(dev, (q_idx_out, _BF16, (B, Tq, H_I, D_I))))
                and workspace.dtype is _U8 and workspace.is_contiguous()
                and workspace.get_device() == dev and kv_new is not None and q_start is not None
                and _rows_good(k_cache, B, D_I, k_cache.seq_stride, dev)
                and _rows_good(kv_cache, B, RLAT, kv_cache.seq_stride, dev))
    except AttributeError:
        good = False
    if not good:
        for rows, width, name in ((k_cache, D_I, "k_cache"), (kv_cache, RLAT, "kv_cache")):
            _refuse_rows(rows, B, width, rows.seq_stride if isinstance(rows, Rows) else 0, dev, name)
        _refuse("dsa_cache_append_rope", dev, (k_pre, (_F32,), None, "k_pre"),
                (kv_new, (_BF16,), (B, Tq, RLAT), "kv_new"), (q_start, (_I32,), (B,), "q_start"),
                (rope, (_F32,), (n_pos, ROPE_DIMS), "rope"), (workspace, (_U8,), None, "workspace"),
                *((t, (dt,), sh, name) for t, dt, sh, name in
                  ((pos, _I32, (B, Tq), "pos"), (n_new, _I32, (B,), "n_new"),
                   (q_pe, _BF16, (B, Tq, H, ROPE_DIMS), "q_pe"),
                   (q_lat, _BF16, (B, Tq, H, RLAT), "q_lat"),
                   (q_idx, _BF16, (B, Tq, H_I, D_I), "q_idx"),
                   (q_idx_out, _BF16, (B, Tq, H_I, D_I), "q_idx_out")) if t is not None))
    code = lib.dsa_cache_append_rope(
        k_pre.data_ptr(), kv_new.data_ptr(), k_cache._p(), kv_cache._p(), q_start.data_ptr(),
        rope.data_ptr(), n_pos, _at(pos), _at(n_new), _at(q_pe), _at(q_lat), H, _at(q_idx),
        _at(q_idx_out), H_I, B, Tq, D_I, kv_style, key_style, eps, workspace.data_ptr(),
        workspace.numel(), raw)
    if code:
        raise DsaError(code, "dsa_cache_append_rope")
    return workspace


def mla_tree_fwd(q_lat, kv: Rows, tree, kv_len, max_kv_len: int, n_draft=None,
                 scale: float = MLA_SCALE, o_lat=None, lse=None, want_lse: bool = True,
                 workspace=None, stream=None):
    """Dense attention of drafted tokens over a latent cache.  q_lat [B,T,H,576] bf16, kv Rows
    (width 576) with the prefix's kv_len[b] rows and then the drafted tokens', tree [B,T]
    int64 (bit j of tree[b,i]: token i sees drafted token j), kv_len [B] int32, n_draft [B]
    int32 drafted tokens that are there (None: T) -> (o_lat [B,T,H,512] bf16, lse [B,T,H]
    float32 or None); outputs of tokens that are not there stay as they were (a new o_lat
    and lse: zeros)."""
    dev = _device(q_lat, "q_lat")
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return mla_tree_fwd(q_lat, kv, tree, kv_len, max_kv_len, n_draft, scale, o_lat, lse,
                                want_lse, workspace, stream)
    raw = _stream_on(dev, stream)
    B, T, H = _queries("mla_tree_fwd", q_lat)
    _ints("mla_tree_fwd", max_kv_len=max_kv_len)
    new = _empty if n_draft is None else _zeros
    if o_lat is None:
        o_lat = new((B, T, H, VLAT), _BF16, dev, stream)
    if lse is None and want_lse:
        lse = new((B, T, H), _F32, dev, stream)
    if workspace is None:
        workspace = _workspace_for(dev, stream, raw, OP_MLA_TREE, B, T, max_kv_len, H, 0)
    try:
        good = (q_lat.dtype is _BF16 and q_lat.is_contiguous() and tree.dtype is _I64
                and tree.shape == (B, T) and tree.is_contiguous() and kv_len.dtype is _I32
                and kv_len.shape == (B,) and kv_len.is_contiguous() and o_lat.dtype is _BF16
                and o_lat.shape == (B, T, H, VLAT) and o_lat.is_contiguous()
                and workspace.dtype is _U8 and workspace.is_contiguous()
                and dev == tree.get_device() == kv_len.get_device() == o_lat.get_device()
                == workspace.get_device()
                and (n_draft is None or _all_good(dev, (n_draft, _I32, (B,))))
                and (lse is None or _all_good(dev, (lse, _F32, (B, T, H))))
                and _rows_good(kv, B, RLAT, max_kv_len, dev))
    except AttributeError:
        good = False
    if not good:
        _refuse_rows(kv, B, RLAT, max_kv_len, dev, "kv")
        _refuse("mla_tree_fwd", dev, (q_lat, (_BF16,), None, "q_lat"), (tree, (_I64,), (B, T), "tree"),
                (kv_len, (_I32,), (B,), "kv_len"), (o_lat, (_BF16,), (B, T, H, VLAT), "o_lat"),
                (workspace, (_U8,), None, "workspace"),
                *((t, (dt,), sh, name) for t, dt, sh, name in
                  ((n_draft, _I32, (B,), "n_draft"), (lse, _F32, (B, T, H), "lse")) if t is not None))
    code = lib.mla_tree_fwd(q_lat.data_ptr(), kv._p(), tree.data_ptr(), kv_len.data_ptr(),
                            _at(n_draft), B, T, H, max_kv_len, scale, o_lat.data_ptr(), _at(lse),
                            workspace.data_ptr(), workspace.numel(), raw)
    if code:
        raise DsaError(code, "mla_tree_fwd")
    return o_lat, lse


def mla_window_fwd(q_lat, kv: Rows, q_start, kv_len, window: int, n_first: int, max_kv_len: int,
                   scale: float = MLA_SCALE, o_lat=None, lse=None, want_lse: bool = True,
                   workspace=None, stream=None):
    """Dense attention with a sliding window: the query at position t = q_start[b] + i sees the
    rows s <= t with s > t - window or s < n_first.  q_lat [B,Tq,H,576] bf16, kv Rows (width
    576), q_start/kv_len [B] int32 -> (o_lat [B,Tq,H,512] bf16, lse [B,Tq,H] float32 or None)."""
    dev = _device(q_lat, "q_lat")
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return mla_window_fwd(q_lat, kv, q_start, kv_len, window, n_first, max_kv_len, scale,
                                  o_lat, lse, want_lse, workspace, stream)
    raw = _stream_on(dev, stream)
    B, Tq, H = _queries("mla_window_fwd", q_lat)
    _ints("mla_window_fwd", window=window, n_first=n_first, max_kv_len=max_kv_len)
    if o_lat is None:
        o_lat = _empty((B, Tq, H, VLAT), _BF16, dev, stream)
    if lse is None and want_lse:
        lse = _empty((B, Tq, H), _F32, dev, stream)
    if workspace is None:
        workspace = _workspace_for(dev, stream, raw, OP_MLA_WINDOW, B, Tq, max_kv_len, H,
                                   min(window + n_first, max_kv_len))
    try:
        good = (q_lat.dtype is _BF16 and q_lat.is_contiguous() and q_start.dtype is _I32
                and q_start.shape == (B,) and q_start.is_contiguous() and kv_len.dtype is _I32
                and kv_len.shape == (B,) and kv_len.is_contiguous() and o_lat.dtype is _BF16
                and o_lat.shape == (B, Tq, H, VLAT) and o_lat.is_contiguous()
                and workspace.dtype is _U8 and workspace.is_contiguous()
                and dev == q_start.get_device() == kv_len.get_device() == o_lat.get_device()
                == workspace.get_device()
                and (lse is None or _all_good(dev, (lse, _F32, (B, Tq, H))))
                and _rows_good(kv, B, RLAT, max_kv_len, dev))
    except AttributeError:
        good = False
    if not good:
        _refuse_rows(kv, B, RLAT, max_kv_len, dev, "kv")
        _refuse("mla_window_fwd", dev, (q_lat, (_BF16,), None, "q_lat"),
                (q_start, (_I32,), (B,), "q_start"), (kv_len, (_I32,), (B,), "kv_len"),
                (o_lat, (_BF16,), (B, Tq, H, VLAT), "o_lat"), (workspace, (_U8,), None, "workspace"),
                *(() if lse is None else ((lse, (_F32,), (B, Tq, H), "lse"),)))
    code = lib.mla_window_fwd(q_lat.data_ptr(), kv._p(), q_start.data_ptr(), kv_len.data_ptr(), B, Tq,
                              H, window, n_first, max_kv_len, scale, o_lat.data_ptr(), _at(lse),
                              workspace.data_ptr(), workspace.numel(), raw)
    if code:
        raise DsaError(code, "mla_window_fwd")
    return o_lat, lse


def mla_window_bwd(q_lat, kv: Rows, q_start, kv_len, window: int, n_first: int, max_kv_len: int,
                   o_lat, lse, d_o, scale: float = MLA_SCALE, dq=None, dkv=None, workspace=None,
                   stream=None):
    """Backward of mla_window_fwd: (dq [B,Tq,H,576] bf16, dkv bf16 like kv's rows [B,S,576])
    from the forward's o_lat and lse and the gradient d_o [B,Tq,H,512] bf16.  kv contiguous.
    Rows 0..kv_len[b]-1 of dkv are written, the rows behind them left as they were (a new
    dkv: zeros)."""
    dev = _device(q_lat, "q_lat")
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return mla_window_bwd(q_lat, kv, q_start, kv_len, window, n_first, max_kv_len, o_lat, lse,
                                  d_o, scale, dq, dkv, workspace, stream)
    raw = _stream_on(dev, stream)
    B, Tq, H = _queries("mla_window_bwd", q_lat)
    _ints("mla_window_bwd", window=window, n_first=n_first, max_kv_len=max_kv_len)
    if not isinstance(kv, Rows) or not _rows_good(kv, B, RLAT, max_kv_len, dev):
        _refuse_rows(kv, B, RLAT, max_kv_len, dev, "kv")
    rows = kv.base.shape
    if dq is None:
        dq = _empty((B, Tq, H, RLAT), _BF16, dev, stream)
    if dkv is None:
        dkv = _zeros(rows, _BF16, dev, stream)
    if workspace is None:
        workspace = _workspace_for(dev, stream, raw, OP_MLA_WINDOW_BWD, B, Tq, max_kv_len, H,
                                   min(window + n_first, max_kv_len))
    try:
        good = (q_lat.dtype is _BF16 and q_lat.is_contiguous() and workspace.dtype is _U8
                and workspace.is_contiguous() and workspace.get_device() == dev
                and q_start is not None and kv_len is not None and o_lat is not None
                and lse is not None and d_o is not None
                and _all_good(dev, (q_start, _I32, (B,)), (kv_len, _I32, (B,)),
                              (o_lat, _BF16, (B, Tq, H, VLAT)), (lse, _F32, (B, Tq, H)),
                              (d_o, _BF16, (B, Tq, H, VLAT)), (dq, _BF16, (B, Tq, H, RLAT)),
                              (dkv, _BF16, rows)))
    except AttributeError:
        good = False
    if not good:
        _refuse("mla_window_bwd", dev, (q_lat, (_BF16,), None, "q_lat"),
                (q_start, (_I32,), (B,), "q_start"), (kv_len, (_I32,), (B,), "kv_len"),
                (o_lat, (_BF16,), (B, Tq, H, VLAT), "o_lat"), (lse, (_F32,), (B, Tq, H), "lse"),
                (d_o, (_BF16,), (B, Tq, H, VLAT), "d_o"), (dq, (_BF16,), (B, Tq, H, RLAT), "dq"),
                (dkv, (_BF16,), rows, "dkv"), (workspace, (_U8,), None, "workspace"))
    code = lib.mla_window_bwd(q_lat.data_ptr(), kv._p(), q_start.data_ptr(), kv_len.data_ptr(), B, Tq,
                              H, window, n_first, max_kv_len, scale, o_lat.data_ptr(), lse.data_ptr(),
                              d_o.data_ptr(), dq.data_ptr(), dkv.data_ptr(), workspace.data_ptr(),
                              workspace.numel(), raw)
    if code:
        raise DsaError(code, "mla_window_bwd")
    return dq, dkv
