"""Latent caches with rotated positions, and dense attention over them, as cases to be measured.

Four operators: the append of new tokens' indexer keys and latent rows to their caches with
the position rotation applied on the way (and to the queries that go with them); attention
of a tree of drafted tokens over a latent cache; attention with a sliding window and a few
first tokens that stay visible; and the latter's backward pass.  Each has a plain form in
elementary torch operations, a call of the framework's own entry point, and a definition in
64 bits.

Sizes are those of the model that the framework serves: 96 heads (8 in its small
configuration), latent rows of 512 + 64, 64 x 128 (or 4 x 64) indexer heads, batches of 16
and 64 requests, sequences of 4096 and 2 x 8192 tokens, chunks of 2048 and 8192, caches of
up to 131072 rows.
"""

import math

import torch

own = False

R, V, ROT, PAGE = 576, 512, 64, 64      # latent row, its value part, its rotated part; rows of a page
SCALE = 1.0 / math.sqrt(128 + 64)
EPS = 1e-5
THETA = 10000.0
HALVES, PAIRS = 1, 2                    # which dims are rotated together: (i, i + 32) or (2i, 2i + 1)
BLOCK = 128                             # queries that the plain window form takes together


def _append(name, B, T, start, heads, index_heads, width, kv_style, key_style, paged, ragged):
    return {"name": name, "op": "append", "B": B, "T": T, "start": start, "heads": heads,
            "index_heads": index_heads, "width": width, "kv_style": kv_style,
            "key_style": key_style, "paged": paged, "ragged": ragged}


def _tree(name, B, T, H, shortest, longest, paged, ragged):
    return {"name": name, "op": "tree", "B": B, "T": T, "H": H, "shortest": shortest,
            "longest": longest, "paged": paged, "ragged": ragged}


def _window(name, op, B, T, H, start, window, first, paged):
    return {"name": name, "op": op, "B": B, "T": T, "H": H, "start": start, "window": window,
            "first": first, "paged": paged}


def listed():
    return [
        # one request's new token
        _append("append_token", 1, 1, 700, 96, 64, 128, PAIRS, HALVES, True, False),
        # 64 requests, up to 4 drafted tokens each, at their depths in the tree
        _append("append_draft64", 64, 4, 900, 96, 64, 128, PAIRS, HALVES, True, True),
        # the second 8192-token chunk of a long prompt
        _append("append_chunk8192", 1, 8192, 8192, 96, 64, 128, PAIRS, HALVES, True, False),
        # one request's next token over a short cache
        _tree("tree_token", 1, 1, 96, 700, 700, True, False),
        # 16 requests, 8 drafted tokens each
        _tree("tree_decode16", 16, 8, 96, 4096, 16384, True, False),
        # next tokens of four requests with long caches
        _tree("tree_long4", 4, 1, 96, 98304, 131072, True, False),
        # odd sizes: trees of up to 33 tokens, 8 heads, prefixes down to nothing
        _tree("tree_ragged", 5, 33, 8, 0, 3001, False, True),
        # next tokens of 64 requests in a local layer
        _window("window_decode64", "window", 64, 1, 96, 9000, 512, 4, True),
        # a 2048-token chunk of a prompt
        _window("window_chunk2048", "window", 1, 2048, 96, 6144, 1024, 4, True),
        # prefill of 2 sequences x 8192 tokens
        _window("window_head8192", "window", 2, 8192, 96, 0, 1024, 16, False),
        # gradients of a small model's batch, sizes that divide by nothing
        _window("window_bwd_ragged", "window_bwd", 3, 301, 8, 0, 77, 3, False),
        # gradients of a training sequence of 4096 tokens
        _window("window_bwd_4096", "window_bwd", 1, 4096, 96, 0, 1024, 4, False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["append", "tree", "tree", "window", "window", "window_bwd"])
    if op == "append":
        B = _log(rng, 1, 64)
        heads, index_heads, width = rng.choice([(96, 64, 128), (8, 4, 64)])
        return {"op": op, "B": B, "T": _log(rng, 1, 8192 // B), "start": _log(rng, 1, 8192) - 1,
                "heads": heads, "index_heads": index_heads, "width": width,
                "kv_style": rng.choice([HALVES, PAIRS]), "key_style": rng.choice([HALVES, PAIRS]),
                "paged": rng.random() < 0.5, "ragged": rng.random() < 0.5}
    H = rng.choice([8, 96, 96, rng.randint(1, 128)])
    if op == "tree":
        B, T = _log(rng, 1, 16), _log(rng, 1, 64)
        longest = _log(rng, 16, min(131072, 524288 // B, 200_000_000 // (B * T * H)))
        return {"op": op, "B": B, "T": T, "H": H, "shortest": rng.randint(0, longest),
                "longest": longest, "paged": rng.random() < 0.5, "ragged": rng.random() < 0.5}
    window, first = _log(rng, 1, 4096), rng.choice([0, 1, 4, 16, 70])
    most = 1_700_000_000 if op == "window" else 400_000_000       # scores
    n = _log(rng, 1, max(1, min(16384 if op == "window" else 4096,
                                most // (H * (window + first + BLOCK)))))
    B = _log(rng, 1, min(64, n))
    return {"op": op, "B": B, "T": n // B, "H": H, "start": rng.choice([0, _log(rng, 1, 8192)]),
            "window": window, "first": first, "paged": op == "window" and rng.random() < 0.5}


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _physical(s, pos):
    """Rows of the flattened store for positions `pos` [B, ...] of each sequence."""
    b = torch.arange(pos.shape[0], device="cuda").view(-1, *[1] * (pos.dim() - 1))
    if s["table"] is None:
        return b * s["capacity"] + pos
    return s["table"].long()[b, pos // PAGE] * PAGE + pos % PAGE


def _rotate(x, cos, sin, style):
    """x [..., 64] by angles whose cos and sin are [..., 32]."""
    if style == HALVES:
        a, b = x[..., :32], x[..., 32:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)


def _append_plain(s):
    B, T = s["k_pre"].shape[:2]
    pos = s["pos"].long()
    cos, sin = s["rope"][pos, :32], s["rope"][pos, 32:]                  # [B, T, 32]
    k = s["k_pre"] - s["k_pre"].mean(2, keepdim=True)
    k = k * torch.rsqrt(k.square().mean(2, keepdim=True) + EPS)
    k = torch.cat([_rotate(k[..., :ROT], cos, sin, s["key_style"]), k[..., ROT:]], 2).to(torch.bfloat16)
    kv = s["kv_new"].float()
    kv = torch.cat([kv[..., :V], _rotate(kv[..., V:], cos, sin, s["kv_style"])], 2).to(torch.bfloat16)
    cos, sin = cos[:, :, None], sin[:, :, None]
    q_pe = _rotate(s["q_pe"].float(), cos, sin, s["kv_style"]).to(torch.bfloat16)
    q_idx = s["q_idx"].float()
    q_idx = torch.cat([_rotate(q_idx[..., :ROT], cos, sin, s["key_style"]), q_idx[..., ROT:]], 3)
    live = torch.arange(T, device="cuda") < s["n_new"].long()[:, None]   # [B, T]
    rows = _physical(s, s["q_start"].long()[:, None] + torch.arange(T, device="cuda"))[live]
    s["k_cache"].view(-1, s["width"])[rows] = k[live]
    s["kv"].view(-1, R)[rows] = kv[live]
    s["q_lat"][..., V:] = torch.where(live[..., None, None], q_pe, s["q_lat"][..., V:])
    s["q_idx_out"][:] = torch.where(live[..., None, None], q_idx.to(torch.bfloat16), s["q_idx_out"])
    return {"k_cache": s["k_cache"], "kv": s["kv"], "q_lat": s["q_lat"], "q_idx": s["q_idx_out"]}


def _attend(z, see, rows):
    """Scores, visibility and value rows [..., keys, 512] -> outputs and log-sum-exps."""
    z = z.masked_fill(~see, -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - top.clamp(min=-1e30))
    total = p.sum(-1, keepdim=True)
    o = p @ rows / total.clamp(min=1e-30)
    return o, (top + torch.log(total)).squeeze(-1)


def _tree_plain(s):
    B, T, H, _ = s["q_lat"].shape
    j = torch.arange(s["longest"] + T, device="cuda")
    kv_len = s["kv_len"].long()[:, None]
    rows = s["kv"].view(-1, R)[_physical(s, j.clamp(max=s["capacity"] - 1).expand(B, -1))].float()
    draft = j - kv_len                                                   # [B, keys]
    bit = (s["tree"][:, :, None] >> draft.clamp(0, 63)[:, None, :]) & 1
    see = (draft < 0)[:, None] | ((draft >= 0) & (draft < T))[:, None] & (bit == 1)
    q = s["q_lat"].float().view(B, T * H, R)
    z = (q @ rows.transpose(1, 2)).view(B, T, H, -1) * SCALE
    o, lse = _attend(z.view(B, T * H, -1), see[:, :, None].expand(-1, -1, H, -1).reshape(B, T * H, -1),
                     rows[..., :V])
    live = (torch.arange(T, device="cuda") < s["n_draft"].long()[:, None])[..., None]
    o = torch.where(live[..., None], o.view(B, T, H, V).to(torch.bfloat16), s["o_lat"])
    return {"o_lat": o, "lse": torch.where(live, lse.view(B, T, H), s["lse"])}


def _window_blocks(s):
    """Queries in blocks: rows [B, n, keys, 576] of each block's keys (the first tokens, then
    those that its windows reach), their positions, visibility [B, n, block, keys], and the
    number of padded queries behind the last."""
    B, T, H, _ = s["q_lat"].shape
    window, first, C = s["window"], s["first"], min(BLOCK, s["q_lat"].shape[1])
    n = -(-T // C)
    t = s["q_start"].long()[:, None, None] + torch.arange(n * C, device="cuda").view(1, n, C)
    near = t[..., :1] - window + 1 + torch.arange(window + C - 1, device="cuda")
    head = torch.arange(first, device="cuda").expand(B, n, first)
    pos = torch.cat([head, near], 2)
    far = torch.arange(pos.shape[2], device="cuda") < first              # keys taken as first tokens
    t4, p4 = t[..., None], pos[:, :, None]
    see = (p4 >= 0) & (p4 <= t4) & ((p4 > t4 - window) & (p4 >= first) | far)
    see = see & (torch.arange(n * C, device="cuda") < T).view(1, n, C, 1)
    rows = s["kv"].view(-1, R)[_physical(s, pos.clamp(0, s["capacity"] - 1))].float()
    return rows, pos, see, n * C - T


def _in_blocks(x, n, pad):
    """[B, T, ...] -> FP32 [B, n, block * ..., last], padded with zeros."""
    x = torch.cat([x.float(), x.new_zeros((x.shape[0], pad, *x.shape[2:])).float()], 1)
    return x.view(x.shape[0], n, -1, x.shape[-1])


def _window_plain(s):
    B, T, H, _ = s["q_lat"].shape
    rows, _, see, pad = _window_blocks(s)
    n, C = see.shape[1:3]
    z = _in_blocks(s["q_lat"], n, pad) @ rows.transpose(2, 3) * SCALE
    see = see[:, :, :, None].expand(-1, -1, -1, H, -1).reshape(B, n, C * H, -1)
    o, lse = _attend(z, see, rows[..., :V])
    return {"o_lat": o.view(B, n * C, H, V)[:, :T].to(torch.bfloat16),
            "lse": lse.view(B, n * C, H)[:, :T]}


def _window_bwd_plain(s):
    B, T, H, _ = s["q_lat"].shape
    rows, pos, see, pad = _window_blocks(s)
    n, C = see.shape[1:3]
    q, d_o, o = (_in_blocks(s[x], n, pad) for x in ("q_lat", "d_o", "o_lat"))
    lse = _in_blocks(s["lse"][..., None], n, pad)
    see = see[:, :, :, None].expand(-1, -1, -1, H, -1).reshape(B, n, C * H, -1)
    p = torch.exp((q @ rows.transpose(2, 3) * SCALE - lse).masked_fill(~see, -math.inf))
    dz = p * (d_o @ rows[..., :V].transpose(2, 3) - (d_o * o).sum(3, keepdim=True)) * SCALE
    dq = (dz @ rows).view(B, n * C, H, R)[:, :T]
    part = dz.transpose(2, 3) @ q                                        # [B, n, keys, 576]
    part[..., :V] += p.transpose(2, 3) @ d_o
    dkv = torch.zeros((B, s["capacity"], R), device="cuda")
    at = pos.clamp(0, s["capacity"] - 1).view(B, -1, 1).expand(-1, -1, R)
    dkv.scatter_add_(1, at, part.view(B, -1, R))                         # unseen rows add zeros
    return {"dq": dq.to(torch.bfloat16), "dkv": dkv.to(torch.bfloat16)}


# ---------------------------------------------------------------------------
# inputs, one pass, work
# ---------------------------------------------------------------------------

def _normal(gen, shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def _store(gen, B, longest, width, paged):
    """A cache of BF16 rows for B sequences of up to `longest` tokens: [B, longest, width], or a
    pool of shuffled pages with its table."""
    if not paged:
        return _normal(gen, (B, longest, width)), None, longest
    pages = -(-longest // PAGE)
    order = torch.randperm(B * pages, generator=gen, device="cuda").to(torch.int32)
    return _normal(gen, (B * pages, PAGE, width)), order.view(B, pages), pages * PAGE


def _rope_table(n):
    i = torch.arange(32, device="cuda", dtype=torch.float64)
    angle = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * THETA ** (-i / 32)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _draft_trees(pick, B, T):
    """Random trees of T tokens: who each token sees (itself and its ancestors, a bit each) and
    its depth."""
    seen, depth = [], []
    for _ in range(B):
        sees, deep = [], []
        for j in range(T):
            parent = int(torch.randint(-1, j, (), generator=pick)) if j else -1
            sees.append((sees[parent] if parent >= 0 else 0) | 1 << j)
            deep.append(deep[parent] + 1 if parent >= 0 else 0)
        seen.append([v - (1 << 64) if v >> 63 else v for v in sees])
        depth.append(deep)
    return torch.tensor(seen, dtype=torch.int64), torch.tensor(depth, dtype=torch.int32)


def _first_rows(s, factor):
    """The first row of each sequence larger than the others, as attention's first tokens are."""
    at = _physical(s, torch.zeros((s["q_lat"].shape[0], 1), dtype=torch.int64, device="cuda"))
    s["kv"].view(-1, R)[at.flatten()] *= factor


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    pick = torch.Generator()
    pick.manual_seed(seed)
    op, B, T = case["op"], case["B"], case["T"]
    s = {"op": op}

    def upto(lo, hi):
        return torch.randint(lo, hi + 1, (B,), generator=pick, dtype=torch.int32)

    def ragged(most):
        return (upto(1, most) if case["ragged"] else torch.full((B,), most, dtype=torch.int32)).cuda()

    if op == "append":
        start = upto(case["start"] // 2, case["start"])
        s["width"], longest = case["width"], case["start"] + T
        s["kv"], s["table"], s["capacity"] = _store(gen, B, longest, R, case["paged"])
        s["k_cache"] = _normal(gen, (*s["kv"].shape[:2], case["width"]))
        s["q_start"] = start.cuda()
        depth = _draft_trees(pick, B, T)[1] if case["ragged"] and T <= 64 else torch.arange(T).int()
        s["pos"] = (start[:, None] + depth).to(torch.int32).contiguous().cuda()
        s["n_new"] = ragged(T)
        s["rope"] = _rope_table(longest)
        s["kv_style"], s["key_style"] = case["kv_style"], case["key_style"]
        s["k_pre"] = _normal(gen, (B, T, case["width"]), 2.0, torch.float32) + 0.5
        s["kv_new"] = _normal(gen, (B, T, R))
        s["q_pe"] = _normal(gen, (B, T, case["heads"], ROT))
        s["q_lat"] = _normal(gen, (B, T, case["heads"], R))
        s["q_idx"] = _normal(gen, (B, T, case["index_heads"], case["width"]))
        s["q_idx_out"] = torch.zeros_like(s["q_idx"])
        return s
    H = case["H"]
    s["q_lat"] = _normal(gen, (B, T, H, R))
    if op == "tree":
        s["longest"] = case["longest"]
        kv_len = upto(case["shortest"], case["longest"])
        s["kv"], s["table"], s["capacity"] = _store(gen, B, case["longest"] + T, R, case["paged"])
        s["tree"] = _draft_trees(pick, B, T)[0].cuda()
        s["kv_len"], s["n_draft"] = kv_len.cuda(), ragged(T)
    else:
        start = upto(case["start"] // 2, case["start"])
        s["window"], s["first"] = case["window"], case["first"]
        s["longest"] = case["start"] + T
        s["kv"], s["table"], s["capacity"] = _store(gen, B, s["longest"], R, case["paged"])
        s["q_start"], s["kv_len"] = start.cuda(), (start + T).cuda()
    _first_rows(s, 2.0)
    s["o_lat"] = torch.zeros((B, T, H, V), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.zeros((B, T, H), device="cuda")
    if op == "window_bwd":                       # what the forward pass left behind
        kept = _window_plain(s)
        s["o_lat"], s["lse"] = kept["o_lat"].contiguous(), kept["lse"].contiguous()
        s["d_o"] = _normal(gen, (B, T, H, V))
        s["dq"] = torch.zeros((B, T, H, R), dtype=torch.bfloat16, device="cuda")
        s["dkv"] = torch.zeros((B, s["capacity"], R), dtype=torch.bfloat16, device="cuda")
    return s


_workspace = None        # one for all calls, as a serving loop on one stream keeps it


def _ws(dsa, need):
    global _workspace
    if _workspace is None or _workspace.numel() < need:
        _workspace = dsa.new_workspace(need)
    return _workspace


def _own(s):
    import sparse_attention_serving_gb300 as dsa
    if "rows" not in s:                          # the handle that a serving loop keeps for its cache
        s["rows"] = dsa.Rows(s["kv"], s["table"])
        if s["op"] == "append":
            s["k_rows"] = dsa.Rows(s["k_cache"], s["table"])
    op, rows = s["op"], s["rows"]
    if op == "append":
        dsa.dsa_cache_append_rope(
            s["k_pre"], s["kv_new"], s["k_rows"], rows, s["q_start"], s["rope"], pos=s["pos"],
            n_new=s["n_new"], q_pe=s["q_pe"], q_lat=s["q_lat"], q_idx=s["q_idx"],
            q_idx_out=s["q_idx_out"], kv_style=s["kv_style"], key_style=s["key_style"], eps=EPS,
            workspace=_ws(dsa, 256))
        return {"k_cache": s["k_cache"], "kv": s["kv"], "q_lat": s["q_lat"], "q_idx": s["q_idx_out"]}
    B, T, H, _ = s["q_lat"].shape
    most = s["longest"] + T if op == "tree" else s["longest"]
    code = {"tree": dsa.OP_MLA_TREE, "window": dsa.OP_MLA_WINDOW, "window_bwd": dsa.OP_MLA_WINDOW_BWD}
    # the last size: the keys that a query may see (window and first tokens)
    span = 0 if op == "tree" else s["window"] + s["first"]
    ws = _ws(dsa, dsa.workspace_bytes(code[op], B, T, most, H, span))
    if op == "tree":
        o, lse = dsa.mla_tree_fwd(s["q_lat"], rows, s["tree"], s["kv_len"], most,
                                  n_draft=s["n_draft"], scale=SCALE, o_lat=s["o_lat"],
                                  lse=s["lse"], workspace=ws)
        return {"o_lat": o, "lse": lse}
    if op == "window":
        o, lse = dsa.mla_window_fwd(s["q_lat"], rows, s["q_start"], s["kv_len"], s["window"],
                                    s["first"], most, scale=SCALE, o_lat=s["o_lat"], lse=s["lse"],
                                    workspace=ws)
        return {"o_lat": o, "lse": lse}
    dq, dkv = dsa.mla_window_bwd(s["q_lat"], rows, s["q_start"], s["kv_len"], s["window"],
                                 s["first"], most, s["o_lat"], s["lse"], s["d_o"], scale=SCALE,
                                 dq=s["dq"], dkv=s["dkv"], workspace=ws)
    return {"dq": dq, "dkv": dkv}


def run(s):
    if own:
        return _own(s)
    plain = {"append": _append_plain, "tree": _tree_plain, "window": _window_plain,
             "window_bwd": _window_bwd_plain}
    return plain[s["op"]](s)


def _seen(start, T, window, first):
    """Keys that T queries from position `start` on see, counted once for each query, and rows
    that any of them sees."""
    pairs = sum(min(t + 1, window) + min(first, max(0, t + 1 - window)) for t in range(start, start + T))
    low = max(0, start + 1 - window)
    return pairs, start + T - low + min(first, low)


def work(case):
    op, B, T = case["op"], case["B"], case["T"]
    if op == "append":
        mean = (1 + T) / 2 if case["ragged"] else T
        q = 4 * ROT * case["heads"] + 4 * case["index_heads"] * case["width"]
        row = 6 * case["width"] + 4 * R + q + 4 * ROT
        turned = ROT * (2 + case["heads"] + case["index_heads"])
        return {"bytes": int(B * mean * row), "flops": int(B * mean * (3 * turned + 8 * case["width"]))}
    H = case["H"]
    out = H * (2 * R + 2 * V + 4)
    if op == "tree":
        rows = (T + 1) / 2 if case["ragged"] else T
        keys = (case["shortest"] + case["longest"]) / 2
        return {"bytes": int(B * (keys * 2 * R + rows * (2 * R + out))),
                "flops": int(2 * B * H * rows * (keys + rows / 2) * (R + V))}
    pairs, rows = _seen(case["start"] * 3 // 4, T, case["window"], case["first"])
    if op == "window":
        return {"bytes": int(B * (rows * 2 * R + T * out)), "flops": int(2 * B * H * pairs * (R + V))}
    # in: queries, rows, outputs, their gradients, log-sum-exps; out: both gradients
    return {"bytes": int(B * ((rows + case["start"] * 3 // 4 + T) * 2 * R + T * H * (4 * R + 4 * V + 4))),
            "flops": int(2 * B * H * pairs * (3 * R + 2 * V))}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _turn(x, angles_cos, angles_sin, style):
    """The rotation as a product with complex numbers."""
    z = torch.complex(angles_cos, angles_sin)
    if style == PAIRS:
        y = torch.view_as_complex(x.unflatten(-1, (32, 2)).contiguous()) * z
        return torch.view_as_real(y).flatten(-2)
    y = torch.complex(x[..., :32].contiguous(), x[..., 32:].contiguous()) * z
    return torch.cat([y.real, y.imag], -1)


def _exact_append(case, s):
    k_cache, kv = s["k_cache"].double(), s["kv"].double()
    q_lat, q_idx = s["q_lat"].double(), s["q_idx_out"].double()
    for b in range(case["B"]):
        n, start = int(s["n_new"][b]), int(s["q_start"][b])
        table = s["rope"][s["pos"][b, :n].long()].double()
        c, r = table[:, :32].contiguous(), table[:, 32:].contiguous()
        x = s["k_pre"][b, :n].double()
        mu = x.sum(1, keepdim=True) / case["width"]
        x = (x - mu) / torch.sqrt(((x - mu) ** 2).sum(1, keepdim=True) / case["width"] + EPS)
        x[:, :ROT] = _turn(x[:, :ROT], c, r, case["key_style"])
        row = s["kv_new"][b, :n].double()
        row[:, V:] = _turn(row[:, V:], c, r, case["kv_style"])
        at = torch.arange(start, start + n, device="cuda")
        if s["table"] is None:
            k_cache[b, at], kv[b, at] = x, row
        else:
            page = s["table"][b].long()[at // PAGE]
            k_cache[page, at % PAGE], kv[page, at % PAGE] = x, row
        q_lat[b, :n, :, V:] = _turn(s["q_pe"][b, :n].double(), c[:, None], r[:, None], case["kv_style"])
        q_idx[b, :n] = s["q_idx"][b, :n].double()
        q_idx[b, :n, :, :ROT] = _turn(q_idx[b, :n, :, :ROT], c[:, None], r[:, None], case["key_style"])
    return {"k_cache": k_cache, "kv": kv, "q_lat": q_lat, "q_idx": q_idx}


def _sequence(s, b, n):
    """The first n rows of sequence b."""
    if s["table"] is None:
        return s["kv"][b, :n].double()
    return s["kv"][s["table"][b].long()].flatten(0, 1)[:n].double()


def _softmax_rows(q, rows, see):
    """q [t, H, 576] over rows [n, 576] that `see` [t, n] lets through."""
    z = torch.einsum("thr,nr->thn", q, rows) * SCALE
    z[~see[:, None].expand_as(z)] = -math.inf
    lse = torch.logsumexp(z, 2)
    p = torch.exp(z - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    return p, lse


def _exact_tree(case, s):
    T = case["T"]
    o, lse = s["o_lat"].double(), s["lse"].double()
    for b in range(case["B"]):
        n, L = int(s["n_draft"][b]), int(s["kv_len"][b])
        rows = _sequence(s, b, L + T)
        see = torch.ones((n, L + T), dtype=torch.bool, device="cuda")
        for i in range(n):
            bits = int(s["tree"][b, i])
            see[i, L:] = torch.tensor([bits >> j & 1 for j in range(T)], dtype=torch.bool)
        p, lse[b, :n] = _softmax_rows(s["q_lat"][b, :n].double(), rows, see)
        o[b, :n] = torch.einsum("thn,nv->thv", p, rows[:, :V])
    return {"o_lat": o, "lse": lse}


def _spans(case, s):
    """(sequence, first and last query of a block, rows that they may see, who sees what)"""
    for b in range(case["B"]):
        start = int(s["q_start"][b])
        for i in range(0, case["T"], 256):
            e = min(case["T"], i + 256)
            t = torch.arange(start + i, start + e, device="cuda")[:, None]
            low = max(0, start + i - case["window"] + 1)
            near = torch.arange(low, start + e, device="cuda")
            at = torch.cat([torch.arange(min(case["first"], low), device="cuda"), near])
            yield b, i, e, at, (at <= t) & ((t - at < case["window"]) | (at < case["first"]))


def _exact_window(case, s):
    o, lse = s["o_lat"].double(), s["lse"].double()
    for b, i, e, at, see in _spans(case, s):
        rows = _sequence(s, b, s["longest"])[at]
        p, lse[b, i:e] = _softmax_rows(s["q_lat"][b, i:e].double(), rows, see)
        o[b, i:e] = torch.einsum("thn,nv->thv", p, rows[:, :V])
    return {"o_lat": o, "lse": lse}


def _exact_window_bwd(case, s):
    dq = torch.zeros((case["B"], case["T"], case["H"], R), dtype=torch.float64, device="cuda")
    dkv = torch.zeros((case["B"], s["capacity"], R), dtype=torch.float64, device="cuda")
    for b, i, e, at, see in _spans(case, s):
        rows = s["kv"][b, at].double()
        q, d_o = s["q_lat"][b, i:e].double(), s["d_o"][b, i:e].double()
        z = torch.einsum("thr,nr->thn", q, rows) * SCALE
        p = torch.exp(z - s["lse"][b, i:e].double()[..., None]) * see[:, None]
        p = torch.where(see[:, None].expand_as(p), p, 0.0)
        D = torch.einsum("thv,thv->th", d_o, s["o_lat"][b, i:e].double())
        dz = p * (torch.einsum("thv,nv->thn", d_o, rows[:, :V]) - D[..., None])
        dq[b, i:e] = SCALE * torch.einsum("thn,nr->thr", dz, rows)
        dkv[b, at] += SCALE * torch.einsum("thn,thr->nr", dz, q)
        dkv[b, at, :V] += torch.einsum("thn,thv->nv", p, d_o)
    return {"dq": dq, "dkv": dkv}


def exact(case, seed):
    if case["op"] != "append" and work(case)["flops"] > 8e12:    # about 20 s at a low FP64 rate
        return None
    s = prepare(case, seed)
    definition = {"append": _exact_append, "tree": _exact_tree, "window": _exact_window,
                  "window_bwd": _exact_window_bwd}
    return definition[case["op"]](case, s)
