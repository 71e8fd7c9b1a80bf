"""The FP8 projection path around the gated DSA step, as cases to be measured.

Three operators: the RMS norm that opens a layer (with the residual's addition, and its
result in E4M3 codes with one scale per 128 values), the quantisation of a projection's
weight (one scale per 128 x 128 block), and the projection itself (a matrix product of
the two kinds of codes).  Each has a plain form in elementary torch operations, a call of
the framework's own entry point, and a definition in 64 bits.

Sizes are those of the model that the framework serves: hidden size 7168, 64 x 128
indexer queries (8192 features), 128 indexer-key and 576 latent features, 96 x 128 gated
outputs (12288), batches of 64 requests and of 2 x 8192 tokens.
"""

import math

import torch

own = False

BLOCK = 128
EPS = 1e-5
E4M3_MAX = 448.0
FLOOR = 2.0 ** -100      # the scale of a block of zeros stays finite and invertible


def _norm(name, n, hid, residual, y):
    return {"name": name, "op": "norm", "n": n, "hid": hid, "residual": residual, "y": y}


def _weight(name, N, K):
    return {"name": name, "op": "weight", "N": N, "K": K}


def _linear(name, M, N, K, out):
    return {"name": name, "op": "linear", "M": M, "N": N, "K": K, "out": out}


def listed():
    return [
        # one request's new token enters a layer
        _norm("norm_token", 1, 7168, True, True),
        # a decode step of 64 requests
        _norm("norm_decode64", 64, 7168, True, True),
        # ragged: an odd number of tokens, a width that ends inside a scale block
        _norm("norm_ragged", 777, 1040, False, False),
        # prefill of 2 sequences x 8192 tokens
        _norm("norm_head8192", 16384, 7168, True, True),
        # loading the latent row's down-projection
        _weight("weight_latent", 576, 7168),
        # loading the output projection
        _weight("weight_oproj", 7168, 12288),
        # one request's indexer queries (64 heads x 128)
        _linear("linear_qidx_token", 1, 8192, 7168, "bf16"),
        # 64 requests' raw indexer keys, FP32 as the cache append takes them
        _linear("linear_kpre_decode64", 64, 128, 7168, "f32"),
        # output projection of 64 requests
        _linear("linear_oproj_decode64", 64, 7168, 12288, "bf16"),
        # latent rows of a 2048-token prefill chunk
        _linear("linear_latent_chunk2048", 2048, 576, 7168, "bf16"),
        # ragged in all three sizes
        _linear("linear_ragged", 777, 1001, 1040, "f32"),
        # output projection of 2 sequences x 8192 tokens
        _linear("linear_oproj_head8192", 16384, 7168, 12288, "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "weight", "linear", "linear"])
    if op == "norm":
        return {"op": op, "n": _log(rng, 1, 16384), "hid": 16 * _log(rng, 4, 448),
                "residual": rng.random() < 0.5, "y": rng.random() < 0.5}
    if op == "weight":
        return {"op": op, "N": _log(rng, 1, 7168), "K": 16 * _log(rng, 4, 768)}
    return {"op": op, "M": _log(rng, 1, 16384), "N": _log(rng, 1, 7168),
            "K": 16 * _log(rng, 4, 768), "out": rng.choice(["bf16", "f32"])}


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _blocks(v, dim):
    """Pad `dim` with zeros to whole blocks and split it into [blocks, 128]."""
    n = v.shape[dim]
    pad = -n % BLOCK
    if pad:
        shape = list(v.shape)
        shape[dim] = pad
        v = torch.cat([v, v.new_zeros(shape)], dim)
    return v.unflatten(dim, (-1, BLOCK))


def _codes(v, scale):
    return (v * (1.0 / scale)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _quant_rows(v):
    """FP32 [n, K] -> E4M3 codes [n, K], scales [n, ceil(K/128)]."""
    b = _blocks(v, 1)
    scale = b.abs().amax(2).clamp(min=FLOOR) / E4M3_MAX
    return _codes(b, scale[:, :, None]).flatten(1)[:, :v.shape[1]].contiguous(), scale


def _quant_blocks(v):
    """FP32 [N, K] -> E4M3 codes [N, K], scales [ceil(N/128), ceil(K/128)]."""
    N, K = v.shape
    b = _blocks(_blocks(v, 1), 0)                    # [nb, 128, kb, 128]
    scale = b.abs().amax((1, 3)).clamp(min=FLOOR) / E4M3_MAX
    codes = _codes(b, scale[:, None, :, None])
    return codes.flatten(2).flatten(0, 1)[:N, :K].contiguous(), scale


def _norm_plain(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["gain"].float()
    codes, scale = _quant_rows(y)
    return codes, scale, h.to(torch.bfloat16), y.to(torch.bfloat16)


def _linear_plain(s):
    K = s["codes"].shape[1]
    N = s["w_codes"].shape[0]
    a = s["codes"].view(torch.float8_e4m3fn).float()
    a = a * s["scale"].repeat_interleave(BLOCK, 1)[:, :K]
    w = s["w_codes"].view(torch.float8_e4m3fn).float()
    w = w * s["w_scale"].repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    return (a @ w.t()).to(s["out"].dtype)


# ---------------------------------------------------------------------------
# inputs, one pass, work
# ---------------------------------------------------------------------------

def _normal(gen, shape, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda") * scale


def _activations(gen, n, width):
    """Rows like a residual stream's: N(0,1), a few channels far larger, and a padded
    token's row of zeros behind the others."""
    x = _normal(gen, (n, width))
    loud = torch.randint(0, width, (max(1, width // 256),), generator=gen, device="cuda")
    x[:, loud] *= 16.0
    if n >= 4:
        x[-1] = 0
    return x.to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = {"op": op}
    if op == "norm":
        n, hid = case["n"], case["hid"]
        s["x"] = _activations(gen, n, hid)
        s["residual"] = _activations(gen, n, hid) if case["residual"] else None
        s["gain"] = (1.0 + _normal(gen, (hid,), 0.1)).to(torch.bfloat16)
        # the buffers that a serving loop keeps for its activations
        s["codes"] = torch.empty((n, hid), dtype=torch.uint8, device="cuda")
        s["scale"] = torch.empty((n, -(-hid // BLOCK)), device="cuda")
        s["residual_out"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["y"] = torch.empty_like(s["x"]) if case["y"] else None
    elif op == "weight":
        s["w"] = _normal(gen, (case["N"], case["K"]), 0.02).to(torch.bfloat16)
        s["codes"] = torch.empty((case["N"], case["K"]), dtype=torch.uint8, device="cuda")
        s["scale"] = torch.empty((-(-case["N"] // BLOCK), -(-case["K"] // BLOCK)), device="cuda")
    else:
        M, N, K = case["M"], case["N"], case["K"]
        codes, s["scale"] = _quant_rows(_activations(gen, M, K).float())
        w_codes, s["w_scale"] = _quant_blocks(_normal(gen, (N, K), 0.02).to(torch.bfloat16).float())
        s["codes"], s["w_codes"] = codes.view(torch.uint8), w_codes.view(torch.uint8)
        s["out"] = torch.empty((M, N), device="cuda",
                               dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
    return s


_workspace = None        # one for all calls, as a serving loop on one stream keeps it


def _ws(dsa, need):
    global _workspace
    if _workspace is None or _workspace.numel() < need:
        _workspace = dsa.new_workspace(need)
    return _workspace


def run(s):
    op = s["op"]
    if own:
        import sparse_attention_serving_gb300 as dsa
        if op == "norm":
            dsa.dsa_rmsnorm_fp8(s["x"], s["gain"], residual=s["residual"], eps=EPS,
                                codes=s["codes"], scale=s["scale"],
                                residual_out=s["residual_out"], y=s["y"])
            codes, scale, h, y = s["codes"], s["scale"], s["residual_out"], s["y"]
        elif op == "weight":
            codes, scale = dsa.dsa_quant_fp8_weight(s["w"], codes=s["codes"], scale=s["scale"])
        else:
            M, K = s["codes"].shape
            N = s["w_codes"].shape[0]
            ws = _ws(dsa, dsa.workspace_bytes(dsa.OP_LINEAR_FP8, M, 1, K, N, 0))
            return {"out": dsa.dsa_linear_fp8(s["codes"], s["scale"], s["w_codes"], s["w_scale"],
                                              out=s["out"], workspace=ws)}
    elif op == "norm":
        codes, scale, h, y = _norm_plain(s)
    elif op == "weight":
        codes, scale = _quant_blocks(s["w"].float())
    else:
        return {"out": _linear_plain(s)}
    # the codes as the values that they stand for (times their scale)
    got = {"codes": codes.view(torch.float8_e4m3fn), "scale": scale}
    if op == "norm":
        if s["residual"] is not None:
            got["residual_out"] = h
        if s["y"] is not None:
            got["y"] = y
    return got


def work(case):
    op = case["op"]
    if op == "norm":
        n, hid = case["n"], case["hid"]
        per = 2 + 1 + (4 if case["residual"] else 0) + (2 if case["y"] else 0)
        return {"bytes": n * hid * per + n * -(-hid // BLOCK) * 4 + 2 * hid, "flops": 6 * n * hid}
    if op == "weight":
        N, K = case["N"], case["K"]
        return {"bytes": 3 * N * K + 4 * -(-N // BLOCK) * -(-K // BLOCK), "flops": 2 * N * K}
    M, N, K = case["M"], case["N"], case["K"]
    kb = -(-K // BLOCK)
    return {"bytes": M * K + N * K + 4 * kb * (M + -(-N // BLOCK))
            + M * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * M * N * K}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _each_block(v, rows):
    """max |v| over blocks of `rows` x 128 of [n, K] (64 bits), spread back over [n, K]'s
    columns and rows, and as it stands."""
    n, K = v.shape
    nb, kb = -(-n // rows), -(-K // BLOCK)
    full = torch.zeros((nb * rows, kb * BLOCK), dtype=torch.float64, device=v.device)
    full[:n, :K] = v.abs()
    top = full.view(nb, rows, kb, BLOCK).permute(0, 2, 1, 3).reshape(nb, kb, -1).max(2).values
    scale = torch.maximum(top, torch.full_like(top, FLOOR)) / E4M3_MAX
    r = torch.arange(n, device=v.device) // rows
    c = torch.arange(K, device=v.device) // BLOCK
    return scale, scale[r][:, c]


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "linear":
        if 2.0 * case["M"] * case["N"] * case["K"] > 4e12:     # about 20 s at a low FP64 rate
            return None
        K = case["K"]
        col = torch.arange(K, device="cuda") // BLOCK
        row = torch.arange(case["N"], device="cuda") // BLOCK
        a = s["codes"].view(torch.float8_e4m3fn).double() * s["scale"].double()[:, col]
        w = s["w_codes"].view(torch.float8_e4m3fn).double() * s["w_scale"].double()[row][:, col]
        return {"out": torch.einsum("mk,nk->mn", a, w)}
    if op == "weight":
        v = s["w"].double()
        scale, spread = _each_block(v, BLOCK)
        return {"codes": v / spread, "scale": scale}
    h = s["x"].double()
    if s["residual"] is not None:
        h += s["residual"].double()
    v = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["hid"] + EPS) * s["gain"].double()
    scale, spread = _each_block(v, 1)
    got = {"codes": v / spread, "scale": scale}
    if s["residual"] is not None:
        got["residual_out"] = h
    if s["y"] is not None:
        got["y"] = v
    return got
