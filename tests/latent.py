"""References in 64 bits for the operators over latent pages, written from the formulas (torch, double)."""
from __future__ import annotations

import math

import torch

ROPE = 64


def rotate(x, rope, positions, interleaved):
    """x [T, H, 64] turned by its positions' rows of the table: every product and sum rounded to fp32."""
    x = x.float()
    c, s = rope[positions, None, :32], rope[positions, None, 32:]
    i = 2 * torch.arange(32) if interleaved else torch.arange(32)
    j = i + 1 if interleaved else i + 32
    out = x.clone()
    a, b = x[..., i], x[..., j]
    out[..., i] = a * c - b * s
    out[..., j] = b * c + a * s
    return out


def norm(c, weight, eps):
    """c [T, dl] in 64 bits: c w / sqrt(mean(c^2) + eps)."""
    c = c.double()
    return c / torch.sqrt((c * c).mean(1, keepdim=True) + eps) * weight.double()


def norm_bound(y, dl):
    """What norm may be off by: the sum of dl squares in fp32 (a lane's dl / 32 in turn and five pairwise: dl / 32 + 5
    roundings of 2^-24), mean, eps, root, reciprocal and two products (a rounding of 2^-24 each), and half a step of bf16."""
    return y.abs() * (2.0 ** -8 + (dl / 32 + 5 + 8) * 2.0 ** -24) + 1e-38


def attention(q, pool, table, lens, page, sm, ok=None):
    """q [B, Tq, Hq, D], pool [nb, page, D] (bf16 values): out [B, Tq, Hq, D - 64] in 64 bits, and what the kernel's roundings
    may add.  ok: [B, positions] whether a position counts (None: all).

    The bound, per output element (n tokens seen, p the probabilities, c the latents, o the output):
      * bf16 output: half a step, 2^-8 |o|;
      * p rounded to bf16, off by 2^-8 of itself at most, divided by the sum of the rounded: 2^-8 sum_t p_t |c_t - o|, with
        another 2^-8 of that for the quotient;
      * ex2.approx (2^-22) of a score in fp32: its argument is within 2^-22 |x| + 2^-21 of the exact one, so p is within
        (|x| 1.45 + 8) 2^-21, and the scores' sums keep 24 bits: each of D / 16 steps loses at most 2^-23 of the sum of
        magnitudes;
      * sums of the value products the same: n / 16 + 2 steps, and as many rescalings and joins.
    """
    B, Tq, Hq, D = q.shape
    dl = D - ROPE
    q = q.double()
    out = torch.zeros(B, Tq, Hq, dl, dtype=torch.float64, device=q.device)
    bound = torch.full_like(out, 1e-30)
    for b in range(B):
        L = int(lens[b])
        if L <= 0:
            continue
        k = pool[table[b, : -(-L // page)].long().clamp(0, pool.shape[0] - 1)].double().flatten(0, 1)[:L]
        k = torch.where(ok[b, :L, None], k, torch.zeros_like(k)) if ok is not None else k
        c = k[:, :dl]
        for i in range(Tq):
            n = L - Tq + 1 + i
            if n <= 0:
                continue
            see = torch.ones(n, dtype=torch.bool, device=q.device) if ok is None else ok[b, :n]
            if not bool(see.any()):
                continue
            x = (q[b, i] @ k[:n].T) * sm
            x = x.masked_fill(~see, -math.inf)
            w = torch.exp(x - x.amax(-1, keepdim=True))
            p = w / w.sum(-1, keepdim=True)
            o = p @ c[:n]
            A = p @ c[:n].abs()
            x = torch.where(see, x, torch.zeros_like(x))
            mag = (q[b, i].abs() @ k[:n].abs().T) * abs(sm)
            dx = D / 16 * 2.0 ** -23 * mag + (x.abs() * 1.45 + 8) * 2.0 ** -21
            dA = (p * dx) @ c[:n].abs() + (p * dx).sum(-1, keepdim=True) * A
            spread = torch.stack([(p[h][:, None] * (c[:n] - o[h]).abs()).sum(0) for h in range(Hq)])
            out[b, i] = o
            bound[b, i] = 2.0 ** -8 * o.abs() + 2.0 ** -8 * (1 + 2.0 ** -7) * spread + dA * (1 + 2.0 ** -7) + \
                (n / 8 + 8) * 2.0 ** -23 * A + 1e-30
    return out, bound
