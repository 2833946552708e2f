"""The latent-cache operators: cases, inputs, plain forms and the framework's calls.

Three operators over pages that hold one latent vector and one rotated key part per token, shared by all heads:
appending tokens (the latent normalised, key and query parts rotated by position), and attention of one token (decode)
or of the last tokens (prefill) of every sequence in its absorbed form.

The pool is bf16 [num_blocks][page][latent + 64]: a row's scores are taken against all of it, its value is the latent.
"""
import math
import random

import torch

own = False

ROPE = 64  # coordinates of the rotated key part
EPS = 1e-6


# ---- cases -----------------------------------------------------------------------------------------------

def listed():
    return [
        # one new token for each of 8 sequences: the append of a decode step (latency)
        {"name": "append_step8", "op": "append", "dl": 512, "page": 64, "hq": 64, "batch": 8, "past_lo": 2000,
         "past_hi": 9000, "new_lo": 1, "new_hi": 1, "pad": 0, "norm": True, "interleaved": True},
        # ragged chunks of several prompts packed into one call with padding behind them, narrow latents
        {"name": "append_ragged", "op": "append", "dl": 256, "page": 32, "hq": 20, "batch": 9, "past_lo": 0,
         "past_hi": 2500, "new_lo": 3, "new_hi": 900, "pad": 5, "norm": True, "interleaved": False},
        # one long prompt's chunk
        {"name": "append_chunk8k", "op": "append", "dl": 512, "page": 16, "hq": 128, "batch": 1, "past_lo": 0,
         "past_hi": 0, "new_lo": 8192, "new_hi": 8192, "pad": 0, "norm": False, "interleaved": True},
        # one short sequence on few heads: the smallest decode call (latency)
        {"name": "decode_tiny", "op": "decode", "dl": 256, "page": 16, "hq": 8, "batch": 1, "lo": 500, "hi": 500},
        # a serving batch of mixed lengths
        {"name": "decode_batch", "op": "decode", "dl": 512, "page": 64, "hq": 64, "batch": 32, "lo": 1024, "hi": 8192},
        # many short sequences, narrow latents
        {"name": "decode_many", "op": "decode", "dl": 256, "page": 32, "hq": 40, "batch": 190, "lo": 1, "hi": 900},
        # all heads of a large layer over long contexts: bandwidth and products close to balance
        {"name": "decode_heads", "op": "decode", "dl": 512, "page": 32, "hq": 128, "batch": 8, "lo": 32768,
         "hi": 32768},
        # few sequences, very long, few heads
        {"name": "decode_long", "op": "decode", "dl": 512, "page": 16, "hq": 32, "batch": 2, "lo": 131072,
         "hi": 131072},
        # a few drafted tokens of a serving batch to verify
        {"name": "prefill_draft4", "op": "prefill", "dl": 512, "page": 64, "hq": 32, "batch": 24, "lo": 1000,
         "hi": 9000, "tq": 4},
        # ragged sequences and an odd number of heads and tokens, narrow latents, some shorter than the chunk
        {"name": "prefill_odd", "op": "prefill", "dl": 256, "page": 32, "hq": 20, "batch": 5, "lo": 40, "hi": 5000,
         "tq": 77},
        # chunks of several prompts
        {"name": "prefill_chunk256", "op": "prefill", "dl": 512, "page": 64, "hq": 64, "batch": 4, "lo": 2000,
         "hi": 8192, "tq": 256},
        # a long prompt's chunk on all heads: the compute-bound end
        {"name": "prefill_long", "op": "prefill", "dl": 512, "page": 16, "hq": 128, "batch": 1, "lo": 16384,
         "hi": 16384, "tq": 1024},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefill"])
    case = {"op": op, "dl": rng.choice([256, 512]), "page": rng.choice([16, 32, 64]),
            "hq": rng.choice([1, 4, 8, 12, 20, 32, 40, 64, 96, 128])}
    if op == "append":
        total = _log(rng, 1, 8000)  # new tokens in all
        batch = min(total, _log(rng, 1, 256))
        each = max(1, total // batch)
        past = _log(rng, 1, 16000)
        case.update(batch=batch, past_lo=rng.choice([0, past // 2]), past_hi=past, new_lo=max(1, each // 2),
                    new_hi=each + rng.randint(0, max(1, each // 4)), pad=rng.choice([0, 0, 1, 7]),
                    norm=rng.random() < 0.5, interleaved=rng.random() < 0.5)
        # past_hi is bounded so that the pool of the whole batch stays small
        case["past_hi"] = max(case["past_lo"], min(case["past_hi"], 400000 // batch))
        case["past_lo"] = min(case["past_lo"], case["past_hi"])
    elif op == "decode":
        cells = _log(rng, 300, 2 * 131072)  # tokens in the cache
        batch = min(_log(rng, 1, 200), cells)
        hi = max(1, min(131072, cells // batch))
        case.update(batch=batch, lo=rng.choice([1, max(1, hi // 2), hi]), hi=hi)
    else:
        tq = _log(rng, 2, 1024)
        hi = _log(rng, 30, 16384)
        batch = max(1, min(_log(rng, 1, 32), int(2e9 / (tq * hi * case["hq"])), int(4e5 / (tq * case["hq"]))))
        case.update(batch=batch, lo=rng.choice([1, max(1, hi // 2), hi]), hi=hi, tq=tq)
    return case


def _spread(lo, hi, n, salt):
    """n whole numbers of [lo, hi], both ends among them where n allows; the same for the same case."""
    if n == 1:
        return [hi]
    r = random.Random(salt * 7919 + lo * 31 + hi * 17 + n)
    return [lo, hi] + [r.randint(lo, hi) for _ in range(n - 2)]


def _lengths(case):
    """(past, new) of each sequence of an append case, or the lengths of an attention case."""
    if case["op"] == "append":
        return _spread(case["past_lo"], case["past_hi"], case["batch"], 1), \
            _spread(case["new_lo"], case["new_hi"], case["batch"], 2)
    return _spread(case["lo"], case["hi"], case["batch"], 3), None


# ---- inputs ----------------------------------------------------------------------------------------------

def _rows(g, n, dl):
    """Latents as a norm leaves them, channels of different strength, and key parts; a few strong tokens."""
    ch = torch.exp(0.4 * torch.randn(dl + ROPE, generator=g, device="cuda"))
    out = torch.empty(n, dl + ROPE, dtype=torch.bfloat16, device="cuda")
    for i in range(0, n, 1 << 18):
        m = min(1 << 18, n - i)
        x = torch.randn(m, dl + ROPE, generator=g, device="cuda") * ch
        x *= 1.0 + 1.5 * (torch.rand(m, 1, generator=g, device="cuda") < 0.02)
        out[i:i + m] = x.to(torch.bfloat16)
    return out


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
    dl, page, hq = case["dl"], case["page"], case["hq"]
    s = {"case": case, "sm_scale": (128 + ROPE) ** -0.5}  # of heads of 128 unrotated and 64 rotated coordinates
    if case["op"] == "append":
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
        # latent and key part side by side, as one projection leaves them; query heads of 128 and 64 coordinates
        s["kv"] = _rows(g, T, dl)
        s["heads"] = torch.randn(T, hq, 128 + ROPE, generator=g, device="cuda").to(torch.bfloat16)
        s["weight"] = torch.exp(0.2 * torch.randn(dl, generator=g, device="cuda")).to(torch.bfloat16) \
            if case["norm"] else None
        s["query"] = torch.zeros(T, hq, dl + ROPE, dtype=torch.bfloat16, device="cuda")  # the attention's input
        inv = 10000.0 ** (-torch.arange(ROPE // 2, dtype=torch.float64, device="cuda") * 2 / ROPE)
        ang = torch.arange(max(ends), dtype=torch.float64, device="cuda")[:, None] * inv[None, :]
        s["rope"] = torch.cat([torch.cos(ang), torch.sin(ang)], 1).to(torch.float32).contiguous()
        s["pool"] = torch.randn(nb, page, dl + ROPE, generator=g, device="cuda").to(torch.bfloat16)
        s["num_blocks"] = nb
        return s
    lens, _ = _lengths(case)
    order.shuffle(lens)
    s["block_table"], nb = _tables(case, lens, g)
    s["num_blocks"] = nb
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["pool"] = _rows(g, nb * page, dl).view(nb, page, dl + ROPE)
    B = case["batch"]
    shape = (B, hq, dl + ROPE) if case["op"] == "decode" else (B, case["tq"], hq, dl + ROPE)
    s["q"] = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
    return s


# ---- plain forms -----------------------------------------------------------------------------------------

def _rotate(x, rope, positions, interleaved):
    """x [T][H][64] in fp32, rotated by position."""
    x, h = x.float(), ROPE // 2
    cs = rope[positions]
    c, sn = cs[:, None, :h], cs[:, None, h:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    a, b = x[..., :h], x[..., h:]
    return torch.cat([a * c - b * sn, b * c + a * sn], -1)


def _plain_append(s):
    case, dl, page = s["case"], s["case"]["dl"], s["case"]["page"]
    live = torch.nonzero(s["slots"] >= 0).squeeze(1)
    slot, pos = s["slots"][live], s["positions"][live]
    inter = case["interleaved"]
    s["query"][live, :, dl:] = _rotate(s["heads"][live, :, 128:], s["rope"], pos, inter).to(torch.bfloat16)
    c = s["kv"][live, :dl].float()
    if s["weight"] is not None:
        c = c * torch.rsqrt((c * c).mean(1, keepdim=True) + EPS) * s["weight"].float()
    k = _rotate(s["kv"][live, None, dl:], s["rope"], pos, inter)[:, 0]
    s["pool"][slot // page, slot % page] = torch.cat([c, k], 1).to(torch.bfloat16)
    return {"q": s["query"][..., dl:], "pool": s["pool"]}


def _plain_attention(s):
    case, q, lens = s["case"], s["q"], s["seq_lens"].long()
    dl, hq, tq = case["dl"], case["hq"], case.get("tq", 1)
    k = s["pool"][s["block_table"].long().clamp(min=0)].float().flatten(1, 2)  # [B][positions][dl + 64]
    B, L = k.shape[0], k.shape[1]
    inside = torch.arange(L, device=q.device)[None, :] < lens[:, None]
    k = torch.where(inside[:, :, None], k, torch.zeros_like(k))
    x = torch.matmul(q.float().view(B, tq * hq, dl + ROPE), k.transpose(1, 2)).mul_(s["sm_scale"]).view(B, tq, hq, L)
    sees = lens[:, None] - tq + torch.arange(1, tq + 1, device=q.device)[None, :]  # positions that each query sees
    hidden = torch.arange(L, device=q.device)[None, None, :] >= sees[:, :, None]
    x.masked_fill_(hidden[:, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, tq * hq, L), k[..., :dl]).view(B, tq, hq, dl)
    o = o / torch.where(total == 0, torch.ones_like(total), total)
    return o.view(*q.shape[:-1], dl).to(torch.bfloat16)


# ---- the framework's calls ---------------------------------------------------------------------------------

_codec = []


def _handle():
    """The handle that a program keeps."""
    if not _codec:
        from rotated_codebook_kv_gb300 import Codec
        _codec.append(Codec(128, 4, 4, 64))
    return _codec[0]


def _own_append(s):
    case, dl = s["case"], s["case"]["dl"]
    kv, q = s["kv"], s["query"][..., dl:]
    _handle().append_latent(kv[:, :dl], kv[:, dl:], s["slots"], s["pool"], case["page"], s["num_blocks"],
                            q=s["heads"][..., 128:], q_out=q, positions=s["positions"], rope=s["rope"],
                            interleaved=case["interleaved"], norm_weight=s["weight"], norm_eps=EPS)
    return {"q": q, "pool": s["pool"]}


def _own_attention(s):
    case, c = s["case"], _handle()
    tq = case.get("tq", 1)
    if "workspace" not in s:  # kept with the sequence plan, as a serving loop keeps it
        s["workspace"] = c.workspace_latent(case["batch"], tq, case["hq"], case["dl"])
        s["out"] = torch.empty(*s["q"].shape[:-1], case["dl"], dtype=torch.bfloat16, device="cuda")
    call = c.decode_attention_latent if case["op"] == "decode" else c.prefill_attention_latent
    return call(s["q"], s["pool"], s["block_table"], s["seq_lens"], case["page"], s["num_blocks"], s["sm_scale"],
                workspace=s["workspace"], out=s["out"])


def run(state):
    append = state["case"]["op"] == "append"
    if own:
        return _own_append(state) if append else _own_attention(state)
    return _plain_append(state) if append else _plain_attention(state)


# ---- the work, and the values in 64 bits ------------------------------------------------------------------

def work(case):
    dl, hq, page = case["dl"], case["hq"], case["page"]
    d = dl + ROPE
    if case["op"] == "append":
        past, new = _lengths(case)
        T = sum(new)
        rows = min(T, max(past) + max(new))  # rows of the rotation's table: positions shared by sequences count once
        return {"bytes": T * (4 * d + 4 * hq * ROPE + 16) + rows * ROPE * 4,
                "flops": T * (3 * (hq + 1) * ROPE + (4 * dl if case["norm"] else 0))}
    lens, _ = _lengths(case)
    tq = case.get("tq", 1)
    pairs = 0
    for n in lens:
        first = max(0, n - tq)  # positions before the chunk
        m = n - first
        pairs += m * first + m * (m + 1) // 2
    by = sum(lens) * 2 * d + 4 * sum(-(-n // page) for n in lens) + case["batch"] * (tq * hq * 2 * (d + dl) + 4)
    return {"bytes": by, "flops": 2 * hq * pairs * (d + dl)}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)


def _exact_turn(x, s):
    half = ROPE // 2
    at = torch.arange(half, device="cuda")
    i, j = (2 * at, 2 * at + 1) if s["case"]["interleaved"] else (at, at + half)
    cs = s["rope"].double()[s["positions"]].unsqueeze(1)
    x = x.double().clone()
    turn = torch.complex(cs[..., :half].contiguous(), cs[..., half:].contiguous())
    z = torch.complex(x[..., i].contiguous(), x[..., j].contiguous()) * turn
    x[..., i], x[..., j] = z.real, z.imag
    return x


def _exact_append(s):
    dl = s["case"]["dl"]
    keep = s["slots"] >= 0
    q = s["query"][..., dl:].double()
    q[keep] = _exact_turn(s["heads"][..., 128:], s)[keep]
    c = s["kv"][:, :dl].double()
    if s["weight"] is not None:
        c = c / torch.sqrt(torch.linalg.vector_norm(c, dim=1, keepdim=True) ** 2 / dl + EPS) * s["weight"].double()
    row = torch.cat([c, _exact_turn(s["kv"][:, None, dl:], s).squeeze(1)], 1)
    pool = s["pool"].double().flatten(0, 1)
    pool[s["slots"][keep]] = row[keep]
    return {"q": q, "pool": pool.view(s["pool"].shape)}


def _exact_attention(s):
    case = s["case"]
    dl, hq, page, tq = case["dl"], case["hq"], case["page"], case.get("tq", 1)
    q = s["q"].double().view(case["batch"], tq, hq, dl + ROPE)
    out = torch.zeros(case["batch"], tq, hq, dl, dtype=torch.float64, device="cuda")
    step = 64  # query tokens at a time
    for b, n in enumerate(s["seq_lens"].tolist()):
        blocks = s["block_table"][b, :-(-n // page)].long()
        k = s["pool"][blocks].double().flatten(0, 1)[:n]
        for t in range(0, tq, step):
            sees = n - tq + 1 + torch.arange(t, min(tq, t + step), device="cuda")
            if int(sees[-1]) < 1:
                continue
            x = torch.einsum("thd,nd->thn", q[b, t:t + step], k) * s["sm_scale"]
            x = x.masked_fill(torch.arange(n, device="cuda")[None, None, :] >= sees[:, None, None], -math.inf)
            w = torch.softmax(x, -1).nan_to_num(0.0)
            out[b, t:t + step] = torch.einsum("thn,nd->thd", w, k[:, :dl])
    return out.view(*s["q"].shape[:-1], dl)
