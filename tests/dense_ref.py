"""Plain 64-bit forms of dense latent attention (drafted trees, windows with first tokens)
and its gradients, with bounds on what the kernels' roundings can add up to.

Per visible row the score is 576 products added in FP32 (an addition off by at most 2^-23 of
the running magnitude, truncation allowed), so z is off by at most
  dz = 580 * 2^-23 * scale * sum |q k| + 2^-21 |z|
(the last term: the scaling, the difference to a reference and the exponential's argument).
p is rounded to BF16 for the value product (2^-8), sums run over n rows in FP32, and the
result is rounded to BF16 once (2^-8)."""
from __future__ import annotations

import math

import torch

SCALE = 1.0 / math.sqrt(192)
HALF = torch.finfo(torch.bfloat16).eps / 2
ADD = 2.0 ** -23


def logical(base, table, b, n):
    """The first n rows of sequence b, 64 bits."""
    if table is None:
        return base[b, :n].double()
    pages = table[b, :-(-n // 64)].long()
    return base[pages].flatten(0, 1)[:n].double()


def window_sees(t, s, window, n_first):
    """t [n, 1], s [m]"""
    return (s <= t) & ((t - s < window) | (s < n_first))


def forward(q, rows, see, scale=SCALE):
    """q [T, H, 576] and rows [n, 576] BF16 or 64-bit, see [T, n] -> o, lse and bounds on the
    kernel's errors of both."""
    q, rows = q.double(), rows.double()
    rows = torch.where(see.any(0)[:, None], rows, 0.0)       # unseen rows may hold anything
    z = torch.einsum("thr,nr->thn", q, rows) * scale
    off = 580 * ADD * scale * torch.einsum("thr,nr->thn", q.abs(), rows.abs()) + z.abs() * 2.0 ** -21
    z = torch.where(see[:, None], z, -math.inf)
    lse = torch.logsumexp(z, 2)
    p = torch.exp(z - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    o = torch.einsum("thn,nv->thv", p, rows[:, :512])
    near = torch.where(see[:, None], off, 0.0).amax(2)       # how far any exponent is off
    size = torch.einsum("thn,nv->thv", p, rows[:, :512].abs())
    n = see.shape[1]
    o_off = (HALF + 2 * near[..., None] + 2 * n * ADD + 2.0 ** -16) * size + HALF * o.abs()
    lse_off = near + (n + 4) * 2.0 ** -24 + lse.abs().clamp(max=1e30) * 2.0 ** -22
    return o, lse, o_off * (1 + 2.0 ** -7), lse_off


def backward(q, rows, see, o, lse, d_o, scale=SCALE):
    """Gradients by the formula from the given o and lse, and bounds on the kernel's errors:
    dq [T, H, 576], dkv [n, 576]."""
    q, rows, o, lse, d_o = (x.double() for x in (q, rows, o, lse, d_o))
    rows = torch.where(see.any(0)[:, None], rows, 0.0)
    z = torch.einsum("thr,nr->thn", q, rows) * scale
    z_off = 580 * ADD * scale * torch.einsum("thr,nr->thn", q.abs(), rows.abs()) + z.abs() * 2.0 ** -21
    lse = torch.where(lse == -math.inf, 0.0, lse)
    p = torch.where(see[:, None], torch.exp(z - lse[..., None]), 0.0)
    p_off = p * (1.05 * z_off + lse.abs()[..., None] * 2.0 ** -22 + 2.0 ** -20)
    v = rows[:, :512]
    dp = torch.einsum("thv,nv->thn", d_o, v) - torch.einsum("thv,thv->th", d_o, o)[..., None]
    dp_off = 516 * ADD * (torch.einsum("thv,nv->thn", d_o.abs(), v.abs())
                          + torch.einsum("thv,thv->th", d_o.abs(), o.abs())[..., None])
    dz = scale * p * dp
    dz_off = scale * (p_off * dp.abs() + p * dp_off) * 1.05
    dz_bf = dz_off + HALF * (dz.abs() + dz_off)               # rounded for the products
    p_bf = p_off + HALF * (p + p_off)
    dq = torch.einsum("thn,nr->thr", dz, rows)
    n, m = see.shape[1], q.shape[0] * q.shape[1]
    dq_off = torch.einsum("thn,nr->thr", dz_bf + 2 * n * ADD * dz.abs(), rows.abs())
    dkv = torch.einsum("thn,thr->nr", dz, q)
    dkv_off = torch.einsum("thn,thr->nr", dz_bf + 2 * m * ADD * dz.abs(), q.abs())
    dkv[:, :512] += torch.einsum("thn,thv->nv", p, d_o)
    dkv_off[:, :512] += torch.einsum("thn,thv->nv", p_bf + 2 * m * ADD * p, d_o.abs())
    grow = 1 + 2.0 ** -7
    return dq, dkv, (dq_off + HALF * dq.abs()) * grow, (dkv_off + HALF * dkv.abs()) * grow


def within(got, ref, off, what):
    got, tiny = got.double(), 2.0 ** -126
    bad = ~((got - ref).abs() <= off + tiny) & ~((got == ref) & torch.isinf(ref))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, e.g. {got[bad][:4].tolist()} "
                           f"for {ref[bad][:4].tolist()}, allowed {off[bad][:4].tolist()}")


def paged(base, gen, spare=3):
    """A contiguous [B, S, W] store as a pool of shuffled pages (S rounded up; the rows behind
    S and the spare pages hold NaN) and its table."""
    B, S, W = base.shape
    pages = -(-S // 64)
    full = torch.full((B, pages * 64, W), math.nan, dtype=base.dtype, device=base.device)
    full[:, :S] = base
    order = torch.randperm(B * pages + spare, generator=gen, device=base.device)[:B * pages]
    pool = torch.full((B * pages + spare, 64, W), math.nan, dtype=base.dtype, device=base.device)
    pool[order] = full.view(B * pages, 64, W)
    return pool, order.view(B, pages).to(torch.int32).contiguous()
