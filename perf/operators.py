"""The paged-cache operators over bf16 and 8-bit pages: cases, inputs, plain forms and the framework's calls.

Four operators: appending rotated keys and values to bf16 pages, the same to e4m3 pages with one scale per
(page, kv head), and attention of one token (decode) or of the last tokens (prefill) over the e4m3 pages.

Pools are [num_blocks][kv heads][page][head dim], scales fp32 [num_blocks][kv heads].  A scale is the least power
of two 2^e (e >= -100) with max |x| <= 448 2^e over the page's rows; a page holds e4m3 codes of x / scale.
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
MIN_EXP = -100


# ---- cases -----------------------------------------------------------------------------------------------

def listed():
    return [
        # one new token for each of 4 long sequences: the append of a decode step, bf16 pages (latency)
        {"name": "append_bf16_step4", "op": "append_bf16", "d": 128, "page": 16, "hq": 64, "hkv": 8, "batch": 4,
         "past_lo": 8000, "past_hi": 16000, "new_lo": 1, "new_hi": 1, "pad": 0, "rot": 128, "interleaved": False},
        # ragged chunks of several prompts packed into one call with padding behind them, bf16 pages
        {"name": "append_bf16_chunks", "op": "append_bf16", "d": 256, "page": 32, "hq": 16, "hkv": 8, "batch": 7,
         "past_lo": 0, "past_hi": 3000, "new_lo": 500, "new_hi": 4000, "pad": 13, "rot": 128, "interleaved": True},
        # one new token for each of 32 sequences: the append of a decode step, 8-bit pages (latency)
        {"name": "append_fp8_step32", "op": "append_fp8", "d": 128, "page": 16, "hq": 32, "hkv": 8, "batch": 32,
         "past_lo": 1024, "past_hi": 8192, "new_lo": 1, "new_hi": 1, "pad": 0, "rot": 128, "interleaved": False},
        # ragged chunks that begin and end inside pages, wide heads, part of the head rotated
        {"name": "append_fp8_ragged", "op": "append_fp8", "d": 256, "page": 32, "hq": 16, "hkv": 8, "batch": 9,
         "past_lo": 1, "past_hi": 2500, "new_lo": 3, "new_hi": 900, "pad": 5, "rot": 64, "interleaved": True},
        # one long prompt's chunk
        {"name": "append_fp8_chunk32k", "op": "append_fp8", "d": 128, "page": 16, "hq": 32, "hkv": 8, "batch": 1,
         "past_lo": 0, "past_hi": 0, "new_lo": 32768, "new_hi": 32768, "pad": 0, "rot": 128, "interleaved": False},
        # one short sequence on few heads: the smallest decode call (latency)
        {"name": "decode_tiny", "op": "decode", "d": 128, "page": 16, "hq": 4, "hkv": 2, "batch": 1, "lo": 512,
         "hi": 512},
        # a serving batch of mixed lengths
        {"name": "decode_paged", "op": "decode", "d": 128, "page": 16, "hq": 32, "hkv": 8, "batch": 32, "lo": 1024,
         "hi": 8192},
        # wide heads, longer pages
        {"name": "decode_wide", "op": "decode", "d": 256, "page": 32, "hq": 16, "hkv": 8, "batch": 8, "lo": 32768,
         "hi": 32768},
        # few sequences, very long
        {"name": "decode_long", "op": "decode", "d": 128, "page": 16, "hq": 64, "hkv": 8, "batch": 4, "lo": 131072,
         "hi": 131072},
        # the last 64 positions of a serving batch (verification of drafted tokens, chunk ends)
        {"name": "prefill_chunk64", "op": "prefill", "d": 128, "page": 16, "hq": 32, "hkv": 8, "batch": 32,
         "lo": 1024, "hi": 8192, "tq": 64},
        # wide heads, a prompt's chunk
        {"name": "prefill_wide", "op": "prefill", "d": 256, "page": 32, "hq": 16, "hkv": 8, "batch": 2, "lo": 5000,
         "hi": 8192, "tq": 1000},
        # a long prompt's chunk: the compute-bound end
        {"name": "prefill_long", "op": "prefill", "d": 128, "page": 16, "hq": 32, "hkv": 8, "batch": 1, "lo": 16384,
         "hi": 16384, "tq": 4096},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append_bf16", "append_fp8", "decode", "prefill"])
    d, page = rng.choice([(128, 16), (128, 32), (256, 16), (256, 32)])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8])
    case = {"op": op, "d": d, "page": page, "hq": hkv * group, "hkv": hkv}
    if op.startswith("append"):
        total = _log(rng, 1, 24000)  # new tokens in all
        batch = min(total, _log(rng, 1, 256))
        each = max(1, total // batch)
        past = _log(rng, 1, 16000)
        case.update(batch=batch, past_lo=rng.choice([0, past // 2]), past_hi=past, new_lo=max(1, each // 2),
                    new_hi=each + rng.randint(0, max(1, each // 4)), pad=rng.choice([0, 0, 1, 7]),
                    rot=rng.choice([0, 32, 64, 80, 128, d]), interleaved=rng.random() < 0.5)
        # past_hi is bounded so that the pool of the whole batch stays small
        case["past_hi"] = max(case["past_lo"], min(case["past_hi"], 400000 // batch))
        case["past_lo"] = min(case["past_lo"], case["past_hi"])
    elif op == "decode":
        cells = _log(rng, 300, 4 * 131072)  # tokens in the cache
        batch = min(_log(rng, 1, 200), cells)
        hi = max(1, min(131072, cells // batch))
        case.update(batch=batch, lo=rng.choice([1, max(1, hi // 2), hi]), hi=hi)
    else:
        tq = _log(rng, 2, 2048)
        hi = _log(rng, 30, 16384)
        batch = max(1, min(_log(rng, 1, 48), int(6e7 / (tq * hi * (d // 128)))))
        case.update(batch=batch, lo=rng.choice([1, max(1, hi // 2), hi]), hi=hi, tq=tq)
    return case


def _spread(lo, hi, n, salt):
    """n whole numbers of [lo, hi], both ends among them where n allows; the same for the same case."""
    if n == 1:
        return [hi]
    r = random.Random(salt * 7919 + lo * 31 + hi * 17 + n)
    mid = [r.randint(lo, hi) for _ in range(n - 2)]
    return [lo, hi] + mid


def _lengths(case):
    """(past, new) of each sequence of an append case, or the lengths of an attention case."""
    if case["op"].startswith("append"):
        return _spread(case["past_lo"], case["past_hi"], case["batch"], 1), \
            _spread(case["new_lo"], case["new_hi"], case["batch"], 2)
    return _spread(case["lo"], case["hi"], case["batch"], 3), None


# ---- inputs ----------------------------------------------------------------------------------------------

def _page_scales(amax):
    """The least power of two 2^e, e >= MIN_EXP, with amax <= 448 2^e (448 = 0.875 * 2^9)."""
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 9 + (m > 0.875), torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)
    return ((e + 127) << 23).view(torch.float32)  # 2^e by its exponent field: ldexp may be off in the last place


def _random_pages(g, nb, hkv, page, d, spread):
    """A pool of e4m3 pages with scales: channels of different strength, some strong tokens."""
    ch = torch.exp(spread * torch.randn(hkv, 1, d, generator=g, device="cuda"))
    codes = torch.empty(nb, hkv, page, d, dtype=torch.uint8, device="cuda")
    scales = torch.empty(nb, hkv, dtype=torch.float32, device="cuda")
    step = max(1, (1 << 28) // (hkv * page * d))
    for i in range(0, nb, step):
        n = min(step, nb - i)
        x = torch.randn(n, hkv, page, d, generator=g, device="cuda") * ch
        x *= 1.0 + 3.0 * (torch.rand(n, 1, page, 1, generator=g, device="cuda") < 0.02)
        s = _page_scales(x.abs().amax(dim=(2, 3)))
        scales[i:i + n] = s
        codes[i:i + n] = (x / s[:, :, None, None]).to(E4M3).view(torch.uint8)
    return codes.view(E4M3), scales


def _tables(case, lens, g):
    """Pages of each sequence on blocks of a random permutation (some blocks are nobody's); unused entries -1."""
    page = case["page"]
    pages = torch.tensor([-(-n // page) for n in lens], device="cuda")
    most = max(1, max(-(-n // page) for n in lens))
    nb = sum(-(-n // page) for n in lens) + 3
    perm = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    start = torch.cumsum(pages, 0) - pages
    col = torch.arange(most, device="cuda")
    table = perm[(start[:, None] + col[None, :]).clamp(max=nb - 1)]
    return torch.where(col[None, :] < pages[:, None], table, torch.full_like(table, -1)).contiguous(), nb


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    order = random.Random(seed)
    d, page, hq, hkv = case["d"], case["page"], case["hq"], case["hkv"]
    s = {"case": case, "sm_scale": d ** -0.5}
    if case["op"].startswith("append"):
        pairs = list(zip(*_lengths(case)))
        order.shuffle(pairs)
        past, new = [p for p, _ in pairs], [n for _, n in pairs]
        ends = [p + n for p, n in zip(past, new)]
        table, nb = _tables(case, ends, g)
        past_t, new_t = torch.tensor(past, device="cuda"), torch.tensor(new, device="cuda")
        total = sum(new)
        seq = torch.repeat_interleave(torch.arange(len(new), device="cuda"), new_t)
        first = torch.cumsum(new_t, 0) - new_t
        pos = past_t[seq] + torch.arange(total, device="cuda") - first[seq]
        slot = table[seq, pos // page].to(torch.int64) * page + pos % page
        pad = torch.full((case["pad"],), -1, dtype=torch.int64, device="cuda")
        s["slots"], s["positions"] = torch.cat([slot, pad]), torch.cat([pos, torch.zeros_like(pad)])
        T = total + case["pad"]
        # the projections of one layer: q, k and v side by side, so rows are strided as a fused projection leaves them
        qkv = torch.randn(T, hq + 2 * hkv, d, generator=g, device="cuda")
        qkv *= torch.exp(0.5 * torch.randn(1, hq + 2 * hkv, d, generator=g, device="cuda"))
        qkv = qkv.to(torch.bfloat16)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_out"] = torch.zeros(T, hq, d, dtype=torch.bfloat16, device="cuda")
        rows = max(ends)
        r = case["rot"]
        inv = 10000.0 ** (-torch.arange(r // 2, dtype=torch.float64, device="cuda") * 2 / max(r, 1))
        ang = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * inv[None, :]
        s["rope"] = torch.cat([torch.cos(ang), torch.sin(ang)], 1).to(torch.float32).contiguous()
        if case["op"] == "append_bf16":
            s["k_pool"] = torch.randn(nb, hkv, page, d, generator=g, device="cuda").to(torch.bfloat16)
            s["v_pool"] = torch.randn(nb, hkv, page, d, generator=g, device="cuda").to(torch.bfloat16)
        else:
            s["k_pool"], s["k_scales"] = _random_pages(g, nb, hkv, page, d, 0.5)
            s["v_pool"], s["v_scales"] = _random_pages(g, nb, hkv, page, d, 0.3)
        s["num_blocks"] = nb
        return s
    lens, _ = _lengths(case)
    order.shuffle(lens)
    s["block_table"], nb = _tables(case, lens, g)
    s["num_blocks"] = nb
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["k_pool"], s["k_scales"] = _random_pages(g, nb, hkv, page, d, 0.5)
    s["v_pool"], s["v_scales"] = _random_pages(g, nb, hkv, page, d, 0.3)
    B = case["batch"]
    shape = (B, hq, d) if case["op"] == "decode" else (B, case["tq"], hq, d)
    s["q"] = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
    return s


# ---- plain forms -----------------------------------------------------------------------------------------

def _rotate(x, rope, positions, r, interleaved):
    """x [T][H][d] in fp32 with its first r coordinates rotated by position."""
    x = x.float()
    if r == 0:
        return x
    cs = rope[positions]
    c, sn = cs[:, None, :r // 2], cs[:, None, r // 2:]
    rot, rest = x[..., :r], x[..., r:]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
        return torch.cat([torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2), rest], -1)
    a, b = rot[..., :r // 2], rot[..., r // 2:]
    return torch.cat([a * c - b * sn, b * c + a * sn, rest], -1)


def _plain_append(s):
    case, slots, positions = s["case"], s["slots"], s["positions"]
    live = torch.nonzero(slots >= 0).squeeze(1)
    slot, pos, page = slots[live], positions[live], case["page"]
    r, inter = case["rot"], case["interleaved"]
    s["q_out"][live] = _rotate(s["q"][live], s["rope"], pos, r, inter).to(torch.bfloat16)
    k = _rotate(s["k"][live], s["rope"], pos, r, inter)
    v = s["v"][live].float()
    block, row = slot // page, slot % page
    if case["op"] == "append_bf16":
        s["k_pool"][block, :, row] = k.to(torch.bfloat16)
        s["v_pool"][block, :, row] = v.to(torch.bfloat16)
        return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    _plain_append_pages(s["k_pool"], s["k_scales"], k, block, row)
    _plain_append_pages(s["v_pool"], s["v_scales"], v, block, row)
    return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"], "k_scales": s["k_scales"],
            "v_scales": s["v_scales"]}


def _plain_append_pages(pool, scales, x, block, row):
    """Rows x of (block, row) into e4m3 pages; a page's earlier rows keep their values under a grown scale."""
    touched, at = torch.unique(block, return_inverse=True)
    n, hkv, page = touched.numel(), pool.shape[1], pool.shape[2]
    amax = torch.zeros(n, hkv, device=x.device).scatter_reduce(
        0, at[:, None].expand(-1, hkv), x.abs().amax(-1), "amax")
    first = torch.full((n,), page, device=x.device).scatter_reduce(0, at, row, "amin")  # rows before it are earlier ones
    need, old = _page_scales(amax), scales[touched]
    new = torch.where((first > 0)[:, None], torch.maximum(old, need), need)
    codes = pool.view(torch.uint8)
    was = codes[touched]
    again = (was.view(E4M3).float() * (old / new)[:, :, None, None]).to(E4M3).view(torch.uint8)
    earlier = torch.arange(page, device=x.device)[None, :] < first[:, None]
    codes[touched] = torch.where(earlier[:, None, :, None], again, was)
    codes[block, :, row] = (x / new[at][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3).view(torch.uint8)
    scales[touched] = new


def _gather(pool, scales, table):
    """fp32 rows [B][kv heads][positions][d] of the sequences' pages."""
    t = table.long().clamp(min=0)
    x = pool.view(torch.uint8)[t].view(E4M3).float() * scales[t][..., None, None]
    B, n, h, p, d = x.shape
    return x.transpose(1, 2).reshape(B, h, n * p, d)


def _plain_attention(s):
    case, q, lens = s["case"], s["q"], s["seq_lens"].long()
    hkv, group, d = case["hkv"], case["hq"] // case["hkv"], case["d"]
    k = _gather(s["k_pool"], s["k_scales"], s["block_table"])
    v = _gather(s["v_pool"], s["v_scales"], s["block_table"])
    B, L = k.shape[0], k.shape[2]
    tq = case.get("tq", 1)
    qr = q.float().reshape(B, tq, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, tq * group, d)
    x = torch.matmul(qr, k.transpose(2, 3)).mul_(s["sm_scale"]).view(B, hkv, tq, group, L)
    sees = lens[:, None] - tq + torch.arange(1, tq + 1, device=q.device)[None, :]  # positions that each query sees
    hidden = torch.arange(L, device=q.device)[None, None, :] >= sees[:, :, None]
    x.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    v = torch.where((torch.arange(L, device=q.device)[None, :] < lens[:, None])[:, None, :, None], v, torch.zeros_like(v))
    o = torch.matmul(p.view(B, hkv, tq * group, L), v).view(B, hkv, tq, group, d)
    o = o / torch.where(total == 0, torch.ones_like(total), total)
    return o.permute(0, 2, 1, 3, 4).reshape(q.shape).to(torch.bfloat16)


# ---- the framework's calls ---------------------------------------------------------------------------------

_codecs = {}


def _codec(d):
    """The handle that a program keeps for a head dim."""
    if d not in _codecs:
        from rotated_codebook_kv_gb300 import Codec
        _codecs[d] = Codec(d, 4, 4, 64)
    return _codecs[d]


def _own_append(s):
    case = s["case"]
    c = _codec(case["d"])
    more = dict(q=s["q"], q_out=s["q_out"], positions=s["positions"], rope=s["rope"] if case["rot"] else None,
                interleaved=case["interleaved"])
    if case["op"] == "append_bf16":
        c.append_kv_bf16(s["k"], s["v"], s["slots"], s["k_pool"], s["v_pool"], case["page"], s["num_blocks"], **more)
        return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    c.append_kv_fp8(s["k"], s["v"], s["slots"], s["k_pool"], s["v_pool"], s["k_scales"], s["v_scales"], case["page"],
                    s["num_blocks"], **more)
    return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"], "k_scales": s["k_scales"],
            "v_scales": s["v_scales"]}


def _own_attention(s):
    case, table = s["case"], s["block_table"]
    c = _codec(case["d"])
    B, hq, hkv, page = case["batch"], case["hq"], case["hkv"], case["page"]
    if "workspace" not in s:  # kept with the sequence plan, as a serving loop keeps it
        if case["op"] == "decode":
            s["splits"] = c.decode_splits_fp8(B, hkv, table.shape[1], page)
            s["workspace"] = c.workspace_fp8(B, hq, s["splits"])
        else:
            s["splits"] = c.prefill_splits_fp8(B, case["tq"], hq, hkv, table.shape[1], page)
            s["workspace"] = c.workspace_fp8(B * case["tq"], hq, s["splits"])
        s["out"] = torch.empty_like(s["q"])
    call = c.decode_attention_fp8 if case["op"] == "decode" else c.prefill_attention_fp8
    return call(s["q"], s["k_pool"], s["v_pool"], s["k_scales"], s["v_scales"], table, s["seq_lens"], hkv, page,
                s["num_blocks"], s["sm_scale"], splits=s["splits"], workspace=s["workspace"], out=s["out"])


def run(state):
    append = state["case"]["op"].startswith("append")
    if own:
        return _own_append(state) if append else _own_attention(state)
    return _plain_append(state) if append else _plain_attention(state)


# ---- the work, and the values in 64 bits ------------------------------------------------------------------

def work(case):
    d, hq, hkv, page = case["d"], case["hq"], case["hkv"], case["page"]
    if case["op"].startswith("append"):
        past, new = _lengths(case)
        T = sum(new)
        cell = 2 if case["op"] == "append_bf16" else 1
        rows = min(T, max(past) + max(new))  # rows of the rotation's table: positions shared by sequences count once
        pages = sum(-(-(n + page - 1) // page) for n in new)
        by = T * (4 * hq * d + 2 * hkv * d * (2 + cell) + 16) + rows * case["rot"] * 4 + \
            (8 * hkv * pages if cell == 1 else 0)
        return {"bytes": by, "flops": 3 * T * (hq + hkv) * case["rot"]}
    lens, _ = _lengths(case)
    tq = case.get("tq", 1)
    cells = sum(lens)
    pages = sum(-(-n // page) for n in lens)
    pairs = 0
    for n in lens:
        first = max(0, n - tq)  # positions before the chunk
        m = n - first
        pairs += m * first + m * (m + 1) // 2
    by = cells * hkv * 2 * d + pages * (8 * hkv + 4) + case["batch"] * (tq * hq * d * 4 + 4)
    return {"bytes": by, "flops": 4 * d * hq * pairs}


def _e4m3_64(x):
    """The nearest e4m3 value of x, ties to even, saturating, in 64 bits."""
    a = x.abs()
    _, e = torch.frexp(a)
    powers = torch.tensor([2.0 ** k for k in range(-9, 140)], dtype=torch.float64, device="cuda")
    step = powers[(e.long() - 4).clamp(min=-9) + 9]
    return (torch.sign(x) * (torch.round(a / step) * step)).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"].startswith("append") else _exact_attention(s)


def _exact_turn(x, s):
    case, r = s["case"], s["case"]["rot"]
    x = x.double().clone()
    if r:
        half = r // 2
        at = torch.arange(half, device="cuda")
        i, j = (2 * at, 2 * at + 1) if case["interleaved"] else (at, at + half)
        cs = s["rope"].double()[s["positions"]].unsqueeze(1)
        turn = torch.complex(cs[..., :half].contiguous(), cs[..., half:].contiguous())
        z = torch.complex(x[..., i].contiguous(), x[..., j].contiguous()) * turn
        x[..., i], x[..., j] = z.real, z.imag
    return x


def _exact_append(s):
    case, page = s["case"], s["case"]["page"]
    keep = s["slots"] >= 0
    slot = s["slots"][keep]
    q = s["q_out"].double()
    q[keep] = _exact_turn(s["q"], s)[keep]
    rows = {"k": _exact_turn(s["k"], s)[keep], "v": s["v"].double()[keep]}
    out = {"q": q}
    for name, x in rows.items():
        pool = s[name + "_pool"].float().double()
        flat = pool.permute(0, 2, 1, 3).reshape(-1, case["hkv"], case["d"])  # by slot
        if case["op"] == "append_bf16":
            flat[slot] = x
            out[name + "_pool"] = flat.view(-1, page, case["hkv"], case["d"]).permute(0, 2, 1, 3).contiguous()
            continue
        scales = s[name + "_scales"].double()
        was = scales.clone()
        fresh = torch.zeros(s["num_blocks"], page, dtype=torch.bool, device="cuda")
        fresh.view(-1)[slot] = True
        hit = fresh.any(1)
        lead = torch.where(hit, fresh.to(torch.int8).argmax(1), 0)  # first new row of each page
        big = torch.zeros(s["num_blocks"] * page, case["hkv"], dtype=torch.float64, device="cuda")
        big[slot] = x.abs().amax(-1)
        big = big.view(-1, page, case["hkv"]).amax(1)
        powers = torch.tensor([2.0 ** e for e in range(MIN_EXP, 130)], dtype=torch.float64, device="cuda")
        need = powers[torch.searchsorted(powers * E4M3_MAX, big.contiguous())]
        grown = torch.where((lead > 0)[:, None], torch.maximum(was, need), need)
        scales = torch.where(hit[:, None], grown, was)
        before = (torch.arange(page, device="cuda")[None, :] < lead[:, None]) & hit[:, None]
        ratio = (was / scales)[:, None, :, None]
        blocks = flat.view(-1, page, case["hkv"], case["d"])
        blocks = torch.where(before[:, :, None, None], _e4m3_64(blocks * ratio), blocks)
        flat = blocks.reshape(-1, case["hkv"], case["d"])
        flat[slot] = _e4m3_64(x / scales[slot // page][..., None])
        out[name + "_pool"] = flat.view(-1, page, case["hkv"], case["d"]).permute(0, 2, 1, 3).contiguous()
        out[name + "_scales"] = scales
    return out


def _exact_attention(s):
    case = s["case"]
    page, hkv, group, tq = case["page"], case["hkv"], case["hq"] // case["hkv"], case.get("tq", 1)
    q = s["q"].double().view(case["batch"], tq, hkv, group, case["d"])
    out = torch.zeros_like(q)
    for b, n in enumerate(s["seq_lens"].tolist()):
        if n == 0:
            continue
        blocks = s["block_table"][b, :-(-n // page)].long()
        sees = n - tq + 1 + torch.arange(tq, device="cuda")
        for h in range(hkv):
            k = (s["k_pool"][:, h].view(torch.uint8)[blocks].view(E4M3).double()
                 * s["k_scales"][blocks, h].double()[:, None, None]).flatten(0, 1)[:n]
            v = (s["v_pool"][:, h].view(torch.uint8)[blocks].view(E4M3).double()
                 * s["v_scales"][blocks, h].double()[:, None, None]).flatten(0, 1)[:n]
            x = torch.einsum("tgd,nd->tgn", q[b, :, h], k) * s["sm_scale"]
            x = x.masked_fill(torch.arange(n, device="cuda")[None, None, :] >= sees[:, None, None], -math.inf)
            w = torch.softmax(x, -1)
            out[b, :, h] = torch.where((sees > 0)[:, None, None], torch.einsum("tgn,nd->tgd", w.nan_to_num(0.0), v), 0.0)
    return out.view(s["q"].shape)
