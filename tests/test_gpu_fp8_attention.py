"""Attention over 8-bit pages (one token, and the last tokens of every sequence) against softmax attention in 64 bits.

The tolerance is derived element by element in paged8.attention from the roundings that the operators declare.
"""
import numpy as np
import pytest
import torch

import paged8 as R
from rotated_codebook_kv_gb300 import Codec, native

pytestmark = pytest.mark.gpu
DEV = "cuda"
_codecs = {}


def _codec(d):
    if d not in _codecs:
        _codecs[d] = Codec(d, 4, 4, 64)
    return _codecs[d]


def case(d, P, Hkv, G, lens, Tq=None, seed=0, spread=0.5, qscale=1.0):
    """Random pages (channels of different strength, scales per page and head), a block table, queries.

    Codes behind a sequence's end and in blocks of nobody are NaN."""
    g = torch.Generator().manual_seed(seed)
    npg = [-(-n // P) for n in lens]
    nb = sum(npg) + 3
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(npg + [1])), -1, dtype=torch.int32)
    codes, scales = [], []
    live = torch.zeros(nb, P, dtype=torch.bool)
    at = 0
    for b, n in enumerate(npg):
        table[b, :n] = perm[at: at + n]
        for i in range(n):
            live[perm[at + i], : max(0, min(P, lens[b] - i * P))] = True
        at += n
    for _ in range(2):
        x = torch.randn(nb, Hkv, P, d, generator=g) * torch.exp(spread * torch.randn(Hkv, 1, d, generator=g))
        amax = x.abs().amax((2, 3))
        s = 2.0 ** torch.ceil(torch.log2(amax / 448))
        c = torch.from_numpy(R.e4m3_codes((x / s[..., None, None]).numpy()))
        c = torch.where(live[:, None, :, None], c, torch.full_like(c, 0x7F))
        codes.append(c)
        scales.append(s.float())
    shape = (len(lens), Hkv * G, d) if Tq is None else (len(lens), Tq, Hkv * G, d)
    q = (torch.randn(shape, generator=g) * qscale).to(torch.bfloat16)
    return dict(q=q, codes=codes, scales=scales, table=table, lens=torch.tensor(lens, dtype=torch.int32), nb=nb, P=P,
                Hkv=Hkv, d=d)


def gpu_pools(c):
    k, v = [x.to(DEV).view(torch.float8_e4m3fn) for x in c["codes"]]
    return k, v, c["scales"][0].to(DEV), c["scales"][1].to(DEV)


def run(c, splits=0, sm=None, **kw):
    codec = _codec(c["d"])
    sm = c["d"] ** -0.5 if sm is None else sm
    call = codec.decode_attention_fp8 if c["q"].dim() == 3 else codec.prefill_attention_fp8
    out = call(c["q"].to(DEV), *gpu_pools(c), c["table"].to(DEV), c["lens"].to(DEV), c["Hkv"], c["P"], c["nb"], sm,
               splits=splits, **kw)
    torch.cuda.synchronize()
    return out


def reference(c, sm=None):
    q = R.bf16(c["q"])
    q4 = q[:, None] if q.ndim == 3 else q
    sm = c["d"] ** -0.5 if sm is None else sm
    out, bound = R.attention(q4, c["codes"][0].numpy(), c["codes"][1].numpy(), c["scales"][0].double().numpy(),
                             c["scales"][1].double().numpy(), c["table"].numpy(), c["lens"].numpy(), c["P"], sm)
    return out.reshape(q.shape), bound.reshape(q.shape)


def check(out, ref, bound):
    err = np.abs(R.bf16(out) - ref)
    assert np.all(np.isfinite(R.bf16(out)))
    worst = float((err / bound).max())
    assert worst <= 1.0, f"error {err.max():.3e}, {worst:.2f} of its bound"
    return worst


DECODE = [
    (128, 16, 2, 8, [1000, 17, 640, 1, 0]),
    (128, 32, 2, 4, [33, 95, 512]),
    (128, 16, 1, 1, [300, 7]),
    (128, 16, 3, 5, [31, 32, 33, 129]),
    (256, 32, 2, 2, [700, 64, 5, 0]),
    (256, 16, 1, 3, [129, 250]),
    (256, 32, 1, 8, [2000]),
]


@pytest.mark.parametrize("d,P,Hkv,G,lens", DECODE)
def test_decode(d, P, Hkv, G, lens):
    c = case(d, P, Hkv, G, lens, seed=d + P + G)
    ref, bound = reference(c)
    for splits in (0, 1, 2, 3, 7):
        check(run(c, splits), ref, bound)
    assert _codec(d).get_status() == 0


PREFILL = [
    (128, 16, 2, 4, [100, 40, 9, 0], 16),
    (128, 32, 1, 8, [70, 33], 33),
    (128, 16, 1, 1, [300], 130),
    (128, 16, 2, 3, [257, 64, 65], 50),
    (256, 16, 1, 2, [90, 31], 40),
    (256, 32, 2, 5, [200, 1], 7),
    (128, 16, 1, 8, [50], 1),
    (128, 16, 1, 2, [5], 20),       # fewer positions than query tokens: the first ones see nothing
]


@pytest.mark.parametrize("d,P,Hkv,G,lens,Tq", PREFILL)
def test_prefill(d, P, Hkv, G, lens, Tq):
    c = case(d, P, Hkv, G, lens, Tq=Tq, seed=d + P + G + Tq)
    ref, bound = reference(c)
    for splits in (0, 1, 2):
        check(run(c, splits), ref, bound)
    assert _codec(d).get_status() == 0


@pytest.mark.parametrize("d", [128, 256])
def test_decode_of_many_sequences(d):
    """More sequences than a block has threads, lengths from 0 on: work dealt out over several stretches of them."""
    g = torch.Generator().manual_seed(d)
    lens = torch.randint(0, 120, (500,), generator=g).tolist()
    lens[0], lens[250], lens[499] = 700, 0, 333
    c = case(d, 16, 1, 2, lens, seed=d)
    ref, bound = reference(c)
    for splits in (0, 1, 2, 9):
        check(run(c, splits), ref, bound)
    assert _codec(d).get_status() == 0


def test_decode_of_empty_sequences():
    c = case(128, 16, 2, 2, [0, 0, 0], seed=1)
    for splits in (1, 2, 5):
        assert torch.all(run(c, splits) == 0)


@pytest.mark.parametrize("d,Hkv,G,B,Tq", [(128, 8, 1, 20, 33), (256, 8, 2, 25, 9)])
def test_prefill_with_units_behind_a_whole_wave(d, Hkv, G, B, Tq):
    """More units than SMs: those that fill waves stay whole, the others are cut."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(1, 160, (B,), generator=g).tolist()
    c = case(d, 16, Hkv, G, lens, Tq=Tq, seed=B)
    ref, bound = reference(c)
    for splits in (0, 1, 3):
        check(run(c, splits), ref, bound)


def test_pool_offsets_past_32_bits():
    """Rows of a pool beyond 4 GiB: appended and attended to."""
    d, P, Hkv = 128, 16, 8
    codec = _codec(d)
    nb = (1 << 32) // (Hkv * P * d) + 40
    kp, vp = [torch.zeros(nb, Hkv, P, d, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2)]
    ks, vs = [torch.ones(nb, Hkv, device=DEV) for _ in range(2)]
    g = torch.Generator().manual_seed(3)
    n = 45
    blocks = torch.tensor([nb - 1, nb - 30, nb - 7], dtype=torch.int32)
    pos = torch.arange(n)
    slots = blocks[pos // P].long() * P + pos % P
    k, v = [torch.randn(n, Hkv, d, generator=g).to(torch.bfloat16) for _ in range(2)]
    codec.append_kv_fp8(k.to(DEV), v.to(DEV), slots.to(DEV), kp, vp, ks, vs, P, nb)
    small = [torch.zeros(3, Hkv, P, d, dtype=torch.uint8).numpy() for _ in range(2)]
    sc = [np.ones((3, Hkv)) for _ in range(2)]
    for x, code, s in ((k, small[0], sc[0]), (v, small[1], sc[1])):
        R.append_fp8(code, s, R.bf16(x), pos.numpy(), np.ones(n, bool), P)
    at = blocks.long().to(DEV)
    assert np.array_equal(kp.view(torch.uint8)[at].cpu().numpy(), small[0])
    assert np.array_equal(vp.view(torch.uint8)[at].cpu().numpy(), small[1])
    lens = torch.tensor([n], dtype=torch.int32)
    for tq in (None, 12):
        q = torch.randn((1, Hkv, d) if tq is None else (1, tq, Hkv, d), generator=g).to(torch.bfloat16)
        call = codec.decode_attention_fp8 if tq is None else codec.prefill_attention_fp8
        out = call(q.to(DEV), kp, vp, ks, vs, blocks[None].to(DEV), lens.to(DEV), Hkv, P, nb, d ** -0.5)
        c = dict(q=q, codes=[torch.from_numpy(x) for x in small], scales=[torch.from_numpy(x) for x in sc],
                 table=torch.arange(3, dtype=torch.int32)[None], lens=lens, nb=3, P=P, Hkv=Hkv, d=d)
        ref, bound = reference(c)
        check(out, ref, bound)
    assert codec.get_status() == 0


@pytest.mark.parametrize("d", [128, 256])
def test_scales_far_apart(d):
    """Pages whose key and value scales differ by many powers of two, one with a zero scale."""
    c = case(d, 16, 2, 4, [200, 90], seed=1)
    g = torch.Generator().manual_seed(2)
    c["scales"][0] *= 2.0 ** torch.randint(-3, 3, c["scales"][0].shape, generator=g)
    c["scales"][1] *= 2.0 ** torch.randint(-9, 9, c["scales"][1].shape, generator=g)
    c["scales"][1][c["table"][0, 1]] = 0.0
    ref, bound = reference(c)
    check(run(c, 1), ref, bound)
    check(run(c, 2), ref, bound)
    # scales that are no powers of two
    c["scales"][0] *= 1.3
    c["scales"][1] *= 0.7
    ref, bound = reference(c)
    check(run(c, 0), ref, bound)


@pytest.mark.parametrize("Tq", [None, 24])
def test_scores_that_grow_and_peak(Tq):
    """Large scores: the running maximum moves often, most probabilities vanish."""
    c = case(128, 16, 1, 4, [400], Tq=Tq, seed=3, qscale=6.0)
    ref, bound = reference(c)
    check(run(c, 0), ref, bound)
    check(run(c, 1), ref, bound)


def test_empty_queries_and_zero_query():
    c = case(128, 16, 2, 2, [40, 0, 12], seed=4)
    c["q"][0] = 0
    ref, bound = reference(c)
    out = run(c)
    check(out, ref, bound)
    assert torch.all(out[1] == 0)
    none = _codec(128).decode_attention_fp8(torch.empty(0, 4, 128, dtype=torch.bfloat16, device=DEV), *gpu_pools(c),
                                            torch.empty(0, 3, dtype=torch.int32, device=DEV),
                                            torch.empty(0, dtype=torch.int32, device=DEV), 2, 16, c["nb"], 0.1)
    assert none.shape == (0, 4, 128)


@pytest.mark.parametrize("d,Tq", [(128, None), (128, 20), (256, None), (256, 20)])
def test_bad_blocks_and_lengths(d, Tq):
    """A bad block counts as hidden; a length past the table is clamped; both set their bits."""
    c = case(d, 16, 2, 4, [200, 100], Tq=Tq, seed=5)
    good = dict(c)
    out0 = run(c)
    c = dict(c, table=c["table"].clone())
    c["table"][0, 2] = c["nb"] + 5
    c["table"][0, 3] = -7
    codec = _codec(d)
    out = run(c)
    assert codec.get_status() == native.TQ_DEVERR_BLOCK_RANGE
    assert np.all(np.isfinite(R.bf16(out))) and torch.equal(out[1], out0[1])
    # what is seen is what the sequence without these pages holds
    if Tq is None:
        keep = [i for i in range(13) if i not in (2, 3)]
        less = dict(good, table=good["table"][:, keep].clone(), lens=torch.tensor([200 - 32, 100], dtype=torch.int32))
        less["table"][1] = good["table"][1, :11]
        ref, bound = reference(less)
        check(out[:1], ref[:1], bound[:1])
    c = dict(good, lens=torch.tensor([100000, 100], dtype=torch.int32))
    run(c, 1)
    assert codec.get_status() & native.TQ_DEVERR_SEQ_RANGE


def test_nan_in_the_cache_and_in_the_query_stays_one():
    c = case(128, 16, 1, 2, [100, 50], seed=6)
    c["codes"][1][c["table"][0, 3], 0, 4, 7] = 0x7F
    out = R.bf16(run(c, 2))
    assert np.all(np.isnan(out[0, :, 7])) and np.all(np.isfinite(np.delete(out[0], 7, axis=1))) and np.all(np.isfinite(out[1]))
    c = case(128, 16, 1, 2, [100, 50], seed=6)
    c["codes"][0][c["table"][1, 1], 0, 4, 7] = 0x7F
    out = R.bf16(run(c, 2))
    assert np.all(np.isnan(out[1])) and np.all(np.isfinite(out[0]))
    c = case(128, 16, 1, 2, [100, 50], seed=6)
    c["q"][0, 1, 5] = float("nan")
    out = R.bf16(run(c, 2))
    assert np.all(np.isnan(out[0, 1])) and np.all(np.isfinite(out[0, 0])) and np.all(np.isfinite(out[1]))


@pytest.mark.parametrize("d,G,Tq,splits", [(128, 2, 4, 1), (128, 2, 4, 3), (256, 1, 7, 2), (128, 4, 100, 1), (128, 8, 33, 2),
                                           (256, 2, 90, 1), (256, 3, 40, 2)])
def test_nan_of_a_later_token_stays_hidden(d, G, Tq, splits):
    """NaN among the last tokens' values and keys: in the rows that see them, and in no others."""
    lens = [200, 131]
    clean = case(d, 16, 2, G, lens, Tq=Tq, seed=11)
    ref, bound = reference(clean)
    c = dict(clean, codes=[x.clone() for x in clean["codes"]])
    want = np.zeros(ref.shape, bool)
    for b, head, back, j in ((0, 0, 1, 5), (0, 1, Tq // 2, d - 1), (0, 1, 2, d - 1), (1, 0, 2, 77), (1, 1, Tq - 1, 64)):
        pos = lens[b] - back
        c["codes"][1][c["table"][b, pos // 16], head, pos % 16, j] = 0xFF if j % 2 else 0x7F
        want[b, Tq - back:, head * G: head * G + G, j] = True
    out = R.bf16(run(c, splits))
    assert np.array_equal(np.isnan(out), want)
    # without the NaN codes the other coordinates are what they were
    assert np.all(np.abs(out - ref)[~want] <= bound[~want])
    c = dict(clean, codes=[x.clone() for x in clean["codes"]])
    pos = lens[1] - 3
    c["codes"][0][c["table"][1, pos // 16], 1, pos % 16, 9] = 0x7F
    out = R.bf16(run(c, splits))
    want = np.zeros(ref.shape, bool)
    want[1, Tq - 3:, G:] = True
    assert np.array_equal(np.isnan(out), want)
    assert np.all(np.abs(out - ref)[~want] <= bound[~want])


@pytest.mark.parametrize("d,Tq", [(128, None), (256, None), (128, 40), (256, 40)])
def test_wait_timeout_reports_and_recovers(d, Tq):
    """With a wait limit of 0 every wait tests its barrier once, the first one as its copies are issued."""
    B, n, P, Hkv = 40, 3000, 16, 2
    npg = -(-n // P)
    g = torch.Generator(device=DEV).manual_seed(7)
    codec = Codec(d, 4, 4, 64)
    pools = codec.alloc_pools_fp8(B * npg, Hkv, P)
    for p in pools[:2]:
        p.view(torch.uint8).copy_(torch.randint(0, 96, p.shape, generator=g, device=DEV))
    table = torch.randperm(B * npg, generator=g, device=DEV).to(torch.int32).view(B, npg)
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    q = torch.randn((B, 4, d) if Tq is None else (B, Tq, 4, d), generator=g, device=DEV).to(torch.bfloat16)
    call = codec.decode_attention_fp8 if Tq is None else codec.prefill_attention_fp8

    def go():
        out = call(q, *pools, table, lens, Hkv, P, B * npg, 0.01, splits=2)
        torch.cuda.synchronize()
        return out

    ref = go()
    assert codec.get_status() == 0
    codec.set_wait_limit(0)
    out = go()
    assert codec.get_status() & native.TQ_DEVERR_TIMEOUT
    assert np.all(np.isfinite(R.bf16(out)))
    codec.set_wait_limit(native.TQ_DEFAULT_WAIT_LIMIT)
    assert torch.equal(go(), ref) and codec.get_status() == 0


def test_two_graphs_with_a_workspace_each_and_another_stream():
    c = case(128, 16, 2, 4, [500, 200], seed=8)
    p = case(128, 16, 2, 4, [500, 200], Tq=30, seed=8)
    codec = _codec(128)
    pools, table, lens = gpu_pools(c), c["table"].to(DEV), c["lens"].to(DEV)
    qd, qp = c["q"].to(DEV), p["q"].to(DEV)
    ppools = gpu_pools(p)
    rd, rp = run(c, 3), run(p, 2)
    wd, wp = codec.workspace_fp8(2, 8, 3), codec.workspace_fp8(60, 8, 2)
    od, op = torch.zeros_like(qd), torch.zeros_like(qp)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        codec.decode_attention_fp8(qd, *pools, table, lens, 2, 16, c["nb"], 128 ** -0.5, splits=3, workspace=wd, out=od)
    with torch.cuda.graph(g2):
        codec.prefill_attention_fp8(qp, *ppools, table, lens, 2, 16, p["nb"], 128 ** -0.5, splits=2, workspace=wp, out=op)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s1):
            g1.replay()
        with torch.cuda.stream(s2):
            g2.replay()
    torch.cuda.synchronize()
    assert torch.equal(od, rd) and torch.equal(op, rp)
    out = codec.decode_attention_fp8(qd, *pools, table, lens, 2, 16, c["nb"], 128 ** -0.5, splits=3, stream=s1)
    s1.synchronize()
    assert torch.equal(out, rd)


def test_refusals():
    c = case(128, 16, 2, 2, [40], seed=9)
    codec = _codec(128)
    pools, table, lens, q = gpu_pools(c), c["table"].to(DEV), c["lens"].to(DEV), c["q"].to(DEV)
    ws = codec.workspace_fp8(1, 4, 3)
    assert codec.workspace_fp8(1, 4, 1).numel() == 0
    ok = (codec.handle, q.data_ptr(), *[x.data_ptr() for x in pools], table.data_ptr(), lens.data_ptr())

    def refused(status, word, B=1, Hq=4, Hkv=2, P=16, maxb=table.shape[1], nb=c["nb"], sm=0.1, splits=3,
                w=ws.data_ptr(), n=ws.numel(), out=q.data_ptr(), first=ok):
        with pytest.raises(native.TQError) as e:
            native.tq_decode_attention_fp8(*first, B, Hq, Hkv, P, maxb, nb, sm, splits, w, n, out, 0)
        assert e.value.status == status and word in str(e.value), str(e.value)

    refused(native.TQ_ERR_UNSUPPORTED, "page_size", P=64)
    refused(native.TQ_ERR_UNSUPPORTED, "1..8", Hq=18)
    refused(native.TQ_ERR_UNSUPPORTED, "1..8", Hq=5)
    refused(native.TQ_ERR_INVALID_ARG, "bad sizes", B=-1)
    refused(native.TQ_ERR_INVALID_ARG, "sm_scale", sm=float("nan"))
    refused(native.TQ_ERR_INVALID_ARG, "workspace", n=ws.numel() - 1)
    refused(native.TQ_ERR_INVALID_ARG, "workspace", w=0)
    refused(native.TQ_ERR_UNSUPPORTED, "splits", splits=1025)
    refused(native.TQ_ERR_UNSUPPORTED, "positions", maxb=1 << 28)
    refused(native.TQ_ERR_UNSUPPORTED, "too large", nb=1 << 40)
    refused(native.TQ_ERR_INVALID_ARG, "NULL", out=0)
    refused(native.TQ_ERR_INVALID_ARG, "misaligned", out=q.data_ptr() + 2)
    with pytest.raises(ValueError):
        codec.decode_attention_fp8(q, *pools, table.long(), lens, 2, 16, c["nb"], 0.1)
    with pytest.raises(ValueError):
        codec.decode_attention_fp8(q, pools[0].float(), *pools[1:], table, lens, 2, 16, c["nb"], 0.1)
    with pytest.raises(ValueError):
        codec.decode_attention_fp8(q.cpu(), *pools, table, lens, 2, 16, c["nb"], 0.1)


def test_refusals_of_sizes_and_of_strided_scratch():
    p = case(128, 16, 2, 2, [40], Tq=20, seed=9)
    codec = _codec(128)
    pools, table, lens, q = gpu_pools(p), p["table"].to(DEV), p["lens"].to(DEV), p["q"].to(DEV)
    head = (codec.handle, q.data_ptr(), *[x.data_ptr() for x in pools], table.data_ptr(), lens.data_ptr())

    def refused(status, word, B=1, tq=20, Hq=4, Hkv=2, splits=1):
        with pytest.raises(native.TQError) as e:
            native.tq_prefill_attention_fp8(*head, B, tq, Hq, Hkv, 16, table.shape[1], p["nb"], 0.1, splits, 0, 0, q.data_ptr(), 0)
        assert e.value.status == status and word in str(e.value), str(e.value)

    refused(native.TQ_ERR_INVALID_ARG, "bad sizes", tq=0)
    refused(native.TQ_ERR_UNSUPPORTED, "too many", B=1 << 20, tq=1 << 12)
    refused(native.TQ_ERR_UNSUPPORTED, "too many", B=1 << 24, tq=20, splits=512)
    refused(native.TQ_ERR_INVALID_ARG, "workspace", splits=2)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device=DEV)[::2]
    with pytest.raises(ValueError):
        codec.prefill_attention_fp8(q, *pools, table, lens, 2, 16, p["nb"], 0.1, splits=2, workspace=ws)
    with pytest.raises(ValueError):
        codec.prefill_attention_fp8(q[0], *pools, table, lens, 2, 16, p["nb"], 0.1)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("sm", [-0.07, 0.0])
def test_score_scales_of_either_sign_and_zero(d, sm):
    for Tq in (None, 2, 24):
        c = case(d, 16, 2, 2, [90, 33], Tq=Tq, seed=12)
        ref, bound = reference(c, sm)
        for splits in (1, 2):
            check(run(c, splits, sm), ref, bound)


@pytest.mark.parametrize("d,P", [(128, 16), (256, 32)])
def test_a_prompt_and_some_tokens_end_to_end(d, P):
    """The set as it is used: append a prompt's chunks and attend to them, then token by token, on both kinds of
    pages.  The 8-bit pages are compared with 64-bit attention over what they hold, the bf16 pages over theirs."""
    codec = _codec(d)
    Hkv, G = 2, 4
    Hq, sm = Hkv * G, d ** -0.5
    nb = 12
    g = torch.Generator().manual_seed(10)
    table = torch.stack([torch.arange(0, 6), torch.arange(6, 12)]).to(torch.int32)
    rope = codec.rope_table(6 * P, d)
    pools8, pools16 = codec.alloc_pools_fp8(nb, Hkv, P), codec.alloc_pools_bf16(nb, Hkv, P)
    lens = [0, 0]
    for new in ([37, 37], [20, 20], [1, 1], [1, 1], [1, 1]):
        pos = torch.cat([torch.arange(a, a + n) for a, n in zip(lens, new)])
        seq = torch.cat([torch.full((n,), b) for b, n in enumerate(new)])
        slots = (table[seq, pos // P].long() * P + pos % P).to(DEV)
        T, tq = pos.numel(), new[0]
        qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=g).to(torch.bfloat16).to(DEV)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        more = dict(q=q, positions=pos.to(DEV), rope=rope)
        q8 = codec.append_kv_fp8(k, v, slots, *pools8, P, nb, **more)
        q16 = codec.append_kv_bf16(k, v, slots, *pools16, P, nb, **more)
        assert torch.equal(q8, q16)
        lens = [a + n for a, n in zip(lens, new)]
        n32 = torch.tensor(lens, dtype=torch.int32, device=DEV)
        c = dict(q=q8.view(2, tq, Hq, d).cpu() if tq > 1 else q8.view(2, Hq, d).cpu(),
                 codes=[p.view(torch.uint8).cpu() for p in pools8[:2]], scales=[s.cpu() for s in pools8[2:]],
                 table=table, lens=n32.cpu(), nb=nb, P=P, Hkv=Hkv, d=d)
        ref, bound = reference(c)
        check(run(c), ref, bound)
        if tq == 1:
            out16 = codec.decode_attention_bf16(q16.view(2, Hq, d), *pools16, table.to(DEV), n32, Hkv, P, nb, sm)
            o16 = R.bf16(out16)
            # an e4m3 key or value is within 2^-4 of its bf16 one (or 2^-10 of the page's scale): the two caches
            # answer alike up to that
            assert np.abs(R.bf16(run(c)) - o16).max() < 0.5 * np.abs(o16).max()
    assert codec.get_status() == 0
