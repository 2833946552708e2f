"""References in 64 bits for the operators over plain bf16 pages and 8-bit pages.

Plain numpy, written from the formulas: rotation by position, page scales and e4m3 codes, attention over the
values that the pages stand for.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
MIN_EXP = -100


def bf16_bits(t):
    import torch
    return t.detach().contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def bf16_to_f64(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def bf16(t):
    """A bf16 tensor's values in 64 bits."""
    return bf16_to_f64(bf16_bits(t))


def _decode_table():
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


E4M3 = _decode_table()


def e4m3_codes(x):
    """Nearest e4m3 codes of x in 64 bits: ties to the even code, saturating, NaN stays one."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), E4M3_MAX)
    grid = E4M3[:127]  # 0 .. 448, ascending
    hi = np.clip(np.searchsorted(grid, np.nan_to_num(a, nan=0.0)), 1, 126)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(x), 127, code)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def page_scale(amax):
    """The least 2^e, e >= -100, with amax <= 448 2^e."""
    e = MIN_EXP
    if amax > 0:
        e = max(MIN_EXP, int(np.ceil(np.log2(amax / E4M3_MAX))) - 1)
        while amax > E4M3_MAX * 2.0 ** e:
            e += 1
    return 2.0 ** e


def rotate(x, pos, rope, interleaved):
    """x [H, d] (64 bits) of the token at pos rotated by its row of the table, products and sums in fp32."""
    r = rope.shape[1]
    out = x.astype(np.float32).copy()
    c, s = rope[pos, : r // 2], rope[pos, r // 2:]
    i = 2 * np.arange(r // 2) if interleaved else np.arange(r // 2)
    j = i + 1 if interleaved else i + r // 2
    a, b = out[:, i].copy(), out[:, j].copy()
    out[:, i] = a * c - b * s
    out[:, j] = b * c + a * s
    return out.astype(np.float64)


def append_fp8(codes, scales, x, slots, ok, page):
    """Rows x [T, H, d] into the pages (codes uint8 [nb, H, P, d], scales fp64 [nb, H]), in place.

    Runs of consecutive slots of one page share a scale; ok: tokens that are written (the others of a run keep
    their place)."""
    T, H, _ = x.shape
    t = 0
    while t < T:
        if slots[t] < 0:
            t += 1
            continue
        blk, o, n = slots[t] // page, slots[t] % page, 1
        while t + n < T and o + n < page and slots[t + n] == slots[t] + n:
            n += 1
        rows = x[t: t + n]
        live = ok[t: t + n]
        for h in range(H):
            y = rows[live, h]
            fin = np.abs(y[np.isfinite(y)])
            need = page_scale(fin.max() if fin.size else 0.0)
            new = max(scales[blk, h], need) if o > 0 else need
            if o > 0 and new > scales[blk, h]:
                codes[blk, h, :o] = e4m3_codes(E4M3[codes[blk, h, :o]] * (scales[blk, h] / new))
            scales[blk, h] = new
            for i in np.nonzero(live)[0]:
                codes[blk, h, o + i] = e4m3_codes(rows[i, h] / new)
        t += n


def attention(q, codes_k, codes_v, ks, vs, table, lens, page, sm):
    """q [B, Tq, Hq, d] in 64 bits -> (out, bound): causal attention of the last Tq positions over e4m3 pages, and
    what the framework's roundings may add.

    The bound, per output element (T tokens seen, p the probabilities, v the values):
      * bf16 output: half a step, 2^-8 |out|;
      * p as two e4m3 terms of fp16(2^8 p): fp16 2^-11 p, the rest of the first term at most 2^-4 of p, the rest of
        the second 2^-4 of that: (2^-8 + 2^-11) p, at least half a subnormal step of the second, 2^-10 / 2^8 of the
        largest p vs: together (2^-8 + 2^-11) A + 2^-18 sum_t max_t(p vs) |code_t| / sum p, A = sum p |v|;
      * ex2.approx (2^-22), fp32 sums and the log2-domain score in fp32: its argument is within 2^-22 |x| + 2^-21
        of the exact one, |x| <= X = max |x|, so e^x is within (X + 4) 2^-21 (twice: p and the sum);
      * q as two e4m3 terms of 2^e q <= 2^8: exact down to 2^-2, then off by at most 2^-10, 2^-17 of the largest
        element: the score by at most 2^-17 max|q| sum_j |k_j| sm;
      * sums of the fp8 products keep 24 bits: each of the d / 16 (scores) and T / 16 + 2 (values; and as many
        rescalings) steps loses at most 2^-23 of the sum of magnitudes.
    """
    B, Tq, Hq, d = q.shape
    Hkv = codes_k.shape[1]
    G = Hq // Hkv
    out = np.zeros(q.shape)
    bound = np.full(q.shape, 1e-30)
    for b in range(B):
        L = int(lens[b])
        npg = -(-L // page)
        for h in range(Hkv):
            blk = table[b, :npg]
            k = (E4M3[codes_k[blk, h]] * ks[blk, h][:, None, None]).reshape(-1, d)[:L]
            cv = E4M3[codes_v[blk, h]].reshape(-1, d)[:L]
            s = np.repeat(vs[blk, h], page)[:L]
            v = cv * s[:, None]
            for i in range(Tq):
                n = L - Tq + 1 + i
                if n <= 0:
                    continue
                for g in range(G):
                    qq = q[b, i, h * G + g]
                    x = (k[:n] @ qq) * sm
                    w = np.exp(x - x.max())
                    p = w / w.sum()
                    o = p @ v[:n]
                    A = p @ np.abs(v[:n])
                    mag = (np.abs(k[:n]) @ np.abs(qq)) * abs(sm)
                    dx = 2.0 ** -17 * np.abs(qq).max() * np.abs(k[:n]).sum(1) * abs(sm) + d / 16 * 2.0 ** -23 * mag + \
                        (np.abs(x) * 1.45 + 8) * 2.0 ** -21
                    dA = (p * dx) @ np.abs(v[:n]) + (p @ dx) * A
                    sub = 2.0 ** -18 * (p * s[:n]).max() * np.abs(cv[:n]).sum(0)
                    out[b, i, h * G + g] = o
                    bound[b, i, h * G + g] = 2.0 ** -8 * (np.abs(o) + A) + 2.0 ** -11 * A + sub + dA + (n / 8 + 4) * 2.0 ** -23 * A + 1e-30
    return out, bound

