"""Latent pages: appending tokens, and attention of one token and of the last tokens of every sequence, against 64 bits.

The attention's tolerance is derived element by element in latent.attention from the roundings that the operators declare.
"""
import numpy as np
import pytest
import torch

import latent as R
from rotated_codebook_kv_gb300 import Codec, native

pytestmark = pytest.mark.gpu
DEV = "cuda"
_codec = []


def codec():
    if not _codec:
        _codec.append(Codec(128, 4, 4, 64))
    return _codec[0]


def case(dl, P, Hq, lens, Tq=None, seed=0, spread=0.4, qscale=1.0, fill=float("nan")):
    """Random latent pages, a block table, queries.  Rows behind a sequence's end and in blocks of nobody hold `fill`."""
    g = torch.Generator().manual_seed(seed)
    D = dl + R.ROPE
    npg = [-(-max(n, 0) // P) for n in lens]
    nb = sum(npg) + 3
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(npg + [1])), -1, dtype=torch.int32)
    live = torch.zeros(nb, P, dtype=torch.bool)
    at = 0
    for b, n in enumerate(npg):
        table[b, :n] = perm[at: at + n]
        for i in range(n):
            live[perm[at + i].long(), : max(0, min(P, lens[b] - i * P))] = True
        at += n
    pool = torch.randn(nb, P, D, generator=g) * torch.exp(spread * torch.randn(D, generator=g))
    pool = torch.where(live[..., None], pool, torch.full_like(pool, fill)).to(torch.bfloat16)
    shape = (len(lens), Hq, D) if Tq is None else (len(lens), Tq, Hq, D)
    q = (torch.randn(shape, generator=g) * qscale).to(torch.bfloat16)
    c = dict(q=q, pool=pool, table=table, lens=torch.tensor(lens, dtype=torch.int32))
    return dict({k: v.to(DEV) for k, v in c.items()}, nb=nb, P=P, dl=dl)


def scale(c):
    return 192 ** -0.5


def run(c, sm=None, **kw):
    call = codec().decode_attention_latent if c["q"].dim() == 3 else codec().prefill_attention_latent
    out = call(c["q"], c["pool"], c["table"], c["lens"], c["P"], c["nb"], scale(c) if sm is None else sm, **kw)
    torch.cuda.synchronize()
    return out


def reference(c, sm=None, ok=None):
    q4 = c["q"][:, None] if c["q"].dim() == 3 else c["q"]
    out, bound = R.attention(q4, c["pool"], c["table"], c["lens"].tolist(), c["P"], scale(c) if sm is None else sm, ok)
    shape = (*c["q"].shape[:-1], c["dl"])
    return out.view(shape), bound.view(shape)


def check(out, ref, bound):
    o = out.double()
    assert bool(torch.isfinite(o).all())
    worst = float(((o - ref).abs() / bound).max()) if o.numel() else 0.0
    assert worst <= 1.0, f"error {float((o - ref).abs().max()):.3e}, {worst:.2f} of its bound"
    return worst


DECODE = [
    (512, 64, 8, [128]),
    (512, 64, 128, [1000, 17, 640, 1, 0]),
    (512, 16, 20, [33, 95, 512, 127, 128, 129]),
    (512, 32, 1, [300, 7]),
    (512, 16, 130, [31, 32, 33, 257]),
    (512, 64, 300, [400]),
    (256, 32, 64, [700, 64, 5, 0]),
    (256, 16, 3, [129, 250]),
    (256, 64, 128, [2000]),
    (256, 32, 260, [63, 65, 1500]),
]


@pytest.mark.parametrize("dl,P,Hq,lens", DECODE)
def test_decode(dl, P, Hq, lens):
    c = case(dl, P, Hq, lens, seed=dl + P + Hq)
    ref, bound = reference(c)
    check(run(c), ref, bound)
    assert codec().get_status() == 0


PREFILL = [
    (512, 64, 32, [100, 40, 9, 0], 4),
    (512, 16, 128, [70, 33], 3),
    (512, 32, 1, [300], 130),
    (512, 16, 20, [257, 64, 65], 50),
    (256, 16, 8, [90, 31], 40),
    (256, 64, 5, [200, 1], 7),
    (256, 32, 100, [500, 129], 3),
    (512, 16, 8, [50], 1),
    (256, 16, 2, [5], 20),          # fewer positions than query tokens: the first ones see nothing
    (512, 64, 150, [260], 2),
]


@pytest.mark.parametrize("dl,P,Hq,lens,Tq", PREFILL)
def test_prefill(dl, P, Hq, lens, Tq):
    c = case(dl, P, Hq, lens, Tq=Tq, seed=dl + P + Hq + Tq)
    ref, bound = reference(c)
    check(run(c), ref, bound)
    assert codec().get_status() == 0


@pytest.mark.parametrize("dl,Hq,n", [(512, 4, 30000), (256, 4, 50001), (512, 128, 5003)])
def test_a_long_sequence_cut_into_many_pieces(dl, Hq, n):
    c = case(dl, 16, Hq, [n], seed=n)
    ref, bound = reference(c)
    check(run(c), ref, bound)


@pytest.mark.parametrize("dl,Hq", [(512, 64), (512, 128), (256, 20), (256, 90)])
def test_sequences_cut_into_several_pieces(dl, Hq):
    """Some ten pieces a sequence, joined row by row; the same call gives the same bits."""
    c = case(dl, 64, Hq, [2500, 2300, 64 * 36, 700, 2501, 2047, 1, 2499], seed=Hq)
    ref, bound = reference(c)
    out = run(c)
    check(out, ref, bound)
    for _ in range(5):
        assert torch.equal(run(c), out)


def test_more_units_than_threads():
    """Row blocks of a few sequences, several of them counted by one thread; lengths below the chunk's."""
    c = case(256, 32, 100, [310, 20, 400], Tq=260, seed=4)
    q, lens = c["q"], c["lens"]
    rows = [0, 1, 100, 239, 240, 258, 259]
    out = run(c)
    for i in rows:  # each query token as the last one of shorter sequences
        one = dict(c, q=q[:, i].contiguous(), lens=(lens - 259 + i).clamp(min=0))
        ref, bound = reference(one)
        check(out[:, i], ref, bound)
    assert codec().get_status() == 0


@pytest.mark.parametrize("Hq,Tq", [(8, None), (70, None), (70, 3)])
def test_outputs_on_16_bytes(Hq, Tq):
    c = case(512, 16, Hq, [500, 77], Tq=Tq, seed=2)
    ref = run(c)
    buf = torch.full((ref.numel() + 16,), 9.0, dtype=torch.bfloat16, device=DEV)
    out = buf[8: 8 + ref.numel()].view(ref.shape)
    assert out.data_ptr() % 32 == 16 and run(c, out=out).data_ptr() == out.data_ptr()
    assert torch.equal(out, ref) and torch.all(buf[:8] == 9) and torch.all(buf[-8:] == 9)


@pytest.mark.parametrize("dl", [256, 512])
def test_decode_of_many_sequences(dl):
    """More sequences than a block has threads, lengths from 0 on."""
    g = torch.Generator().manual_seed(dl)
    lens = torch.randint(0, 300, (500,), generator=g).tolist()
    lens[0], lens[250], lens[499] = 1700, 0, 333
    c = case(dl, 16, 4, lens, seed=dl)
    ref, bound = reference(c)
    check(run(c), ref, bound)
    assert codec().get_status() == 0


def test_empty_sequences_and_batches():
    c = case(512, 16, 20, [0, 0, 0], seed=1)
    assert torch.all(run(c) == 0)
    c = case(256, 16, 20, [0, 0], Tq=9, seed=1)
    assert torch.all(run(c) == 0)
    none = codec().decode_attention_latent(torch.empty(0, 4, 576, dtype=torch.bfloat16, device=DEV), torch.zeros(1, 16, 576, dtype=torch.bfloat16, device=DEV),
                                           torch.empty(0, 3, dtype=torch.int32, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV), 16, 1, 0.1)
    assert none.shape == (0, 4, 512)
    assert codec().get_status() == 0


@pytest.mark.parametrize("dl,Hq,B,Tq", [(512, 20, 30, 33), (256, 12, 60, 40)])
def test_prefill_of_many_units(dl, Hq, B, Tq):
    """More units than pairs of SMs, some cut at the shares' borders."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(1, 400, (B,), generator=g).tolist()
    c = case(dl, 32, Hq, lens, Tq=Tq, seed=B)
    ref, bound = reference(c)
    check(run(c), ref, bound)


@pytest.mark.parametrize("Tq", [None, 24])
@pytest.mark.parametrize("dl", [256, 512])
def test_scores_that_grow_and_peak(dl, Tq):
    """Large scores: the running maximum moves often, most probabilities vanish."""
    c = case(dl, 16, 8, [900], Tq=Tq, seed=3, qscale=8.0)
    ref, bound = reference(c)
    check(run(c), ref, bound)
    # scores that rise along the sequence, so that every tile is the largest so far
    ramp = torch.linspace(0.01, 4.0, 900, device=DEV)
    for i, blk in enumerate(c["table"][0].tolist()):
        n = min(16, 900 - 16 * i)
        c["pool"][blk, :n] = (c["q"].reshape(-1, c["dl"] + 64)[0] * ramp[16 * i: 16 * i + n, None] / 8).to(torch.bfloat16)
    ref, bound = reference(c)
    check(run(c), ref, bound)


@pytest.mark.parametrize("sm", [-0.07, 0.0])
@pytest.mark.parametrize("Tq", [None, 5])
def test_score_scales_of_either_sign_and_zero(sm, Tq):
    c = case(512, 32, 20, [290, 33], Tq=Tq, seed=12)
    ref, bound = reference(c, sm)
    check(run(c, sm), ref, bound)


@pytest.mark.parametrize("dl,Tq", [(512, None), (512, 20), (256, None), (256, 20)])
def test_bad_blocks_and_lengths(dl, Tq):
    """A bad block counts as hidden; a length past the table is clamped; both set their bits."""
    c = case(dl, 16, 4, [400, 100], Tq=Tq, seed=5)
    out0 = run(c)
    bad = dict(c, table=c["table"].clone())
    bad["table"][0, 2] = c["nb"] + 5
    bad["table"][0, 13] = -7
    ok = torch.ones(2, 400, dtype=torch.bool, device=DEV)
    ok[0, 32:48] = ok[0, 13 * 16: 14 * 16] = False
    ref, bound = reference(dict(c), ok=ok)
    out = run(bad)
    assert codec().get_status() == native.TQ_DEVERR_BLOCK_RANGE
    check(out, ref, bound)
    assert torch.equal(out[1], out0[1])
    run(dict(c, lens=torch.tensor([100000, 100], dtype=torch.int32, device=DEV), table=c["table"].clamp(min=0)))
    assert codec().get_status() & native.TQ_DEVERR_SEQ_RANGE
    out = run(dict(c, lens=torch.tensor([-3, 100], dtype=torch.int32, device=DEV)))
    assert torch.all(out[0] == 0) and codec().get_status() == 0


def test_every_block_bad():
    c = case(512, 16, 4, [100], seed=5)
    out = run(dict(c, table=torch.full_like(c["table"], -1)))
    assert torch.all(out == 0) and codec().get_status() == native.TQ_DEVERR_BLOCK_RANGE


@pytest.mark.parametrize("bits", [0x7FC0, 0x7F80, 0xFF80, 0xFFFF])
@pytest.mark.parametrize("dl,Hq,Tq,j", [(512, 4, 7, 5), (512, 20, 20, 511), (256, 8, 40, 255), (512, 64, 3, 300), (256, 1, 100, 0),
                                        (512, 4, 7, 540)])
def test_what_is_not_finite_in_a_later_token_stays_hidden(dl, Hq, Tq, j, bits):
    """NaN and infinities among the last tokens' rows: in the query tokens that see them, and in no others."""
    lens = [300, 131]
    clean = case(dl, 16, Hq, lens, Tq=Tq, seed=11)
    ref, bound = reference(clean)
    c = dict(clean, pool=clean["pool"].clone())
    first = []
    for b, back in ((0, 1), (1, Tq - 1)):
        pos = lens[b] - back
        c["pool"][int(c["table"][b, pos // 16]), pos % 16, j] = torch.tensor(bits, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).item() \
            if bits != 0xFFFF else float("nan")
        first.append(Tq - back)
    out = run(c).double()
    for b in range(2):
        f = first[b]
        clear = out[b, :f]
        assert bool(torch.isfinite(clear).all())
        assert bool(((clear - ref[b, :f]).abs() <= bound[b, :f]).all())
        seen = out[b, f:]
        if j < dl and bits in (0x7FC0, 0xFFFF):
            assert bool(torch.isnan(seen).all())
        elif j < dl:
            assert bool(torch.isnan(seen[..., j]).all())
    assert codec().get_status() == 0


@pytest.mark.parametrize("dl,Hq,Tq", [(512, 20, 40), (256, 1, 50)])
def test_what_is_not_finite_reaches_across_pieces(dl, Hq, Tq):
    """A long sequence cut into many pieces, NaN early (every row sees it) or among its last tokens."""
    n = 6000
    clean = case(dl, 16, Hq, [n], Tq=Tq, seed=13)
    ref = run(clean)
    for pos, first in ((17, 0), (n - 5, Tq - 5), (n - Tq // 2, Tq - Tq // 2)):
        c = dict(clean, pool=clean["pool"].clone())
        c["pool"][int(c["table"][0, pos // 16]), pos % 16, 9] = float("nan")
        out = run(c)
        assert bool(torch.isnan(out[0, first:]).all())
        assert torch.equal(out[0, :first], ref[0, :first])


def test_nan_in_a_query_stays_in_its_row():
    c = case(512, 16, 4, [100, 50], seed=6)
    c["q"][0, 1, 5] = float("nan")
    out = run(c)
    assert bool(torch.isnan(out[0, 1]).all())
    out[0, 1] = 0
    assert bool(torch.isfinite(out.float()).all())


def test_values_near_the_largest():
    """Latents close to bf16's largest number: sums of probabilities times them must not overflow before the division."""
    c = case(512, 16, 4, [700], seed=7)
    c["q"][..., :512] = 0
    live = torch.isfinite(c["pool"].float())
    big = torch.where(torch.rand(c["pool"].shape, device=DEV) < 0.5, 2.9e38, 3.0e38).to(torch.bfloat16)
    c["pool"][..., :512] = torch.where(live[..., :512], big[..., :512], c["pool"][..., :512])
    ref, bound = reference(c)
    check(run(c), ref, bound)


def test_pool_offsets_past_32_bits():
    """Rows of a pool beyond 4 GiB: appended and attended to."""
    dl, P, Hq = 512, 64, 8
    nb = (1 << 32) // (P * 576 * 2) + 40
    pool = codec().alloc_pool_latent(nb, P, dl)
    g = torch.Generator().manual_seed(3)
    n = 145
    blocks = torch.tensor([nb - 1, nb - 30, nb - 7], dtype=torch.int32)
    pos = torch.arange(n)
    slots = blocks[pos // P].long() * P + pos % P
    rows = torch.randn(n, 576, generator=g).to(torch.bfloat16).to(DEV)
    codec().append_latent(rows[:, :dl], rows[:, dl:], slots.to(DEV), pool, P, nb)
    got = pool[blocks.long().to(DEV)].flatten(0, 1)
    assert torch.equal(got[:n], rows) and torch.all(got[n:] == 0)
    for tq in (None, 12):
        q = torch.randn((1, Hq, 576) if tq is None else (1, tq, Hq, 576), generator=g).to(torch.bfloat16).to(DEV)
        c = dict(q=q, pool=pool, table=blocks[None].to(DEV), lens=torch.tensor([n], dtype=torch.int32, device=DEV), nb=nb, P=P, dl=dl)
        ref, bound = reference(c)
        check(run(c), ref, bound)
    assert codec().get_status() == 0


@pytest.mark.parametrize("dl,Hq,Tq", [(512, 4, None), (256, 4, None), (512, 100, None), (256, 100, None), (512, 4, 40), (256, 4, 40),
                                      (512, 4, 9), (256, 4, 9)])
def test_wait_timeout_reports_and_recovers(dl, Hq, Tq):
    """With a wait limit of 0 every wait tests its barrier once, the first one as its copies are issued."""
    own = Codec(128, 4, 4, 64)
    c = case(dl, 16, Hq, [3000] * 30, Tq=Tq, seed=7)

    def go():
        call = own.decode_attention_latent if Tq is None else own.prefill_attention_latent
        out = torch.full((*c["q"].shape[:-1], dl), float("nan"), dtype=torch.bfloat16, device=DEV)
        call(c["q"], c["pool"], c["table"], c["lens"], 16, c["nb"], 0.01, out=out)
        torch.cuda.synchronize()
        return out

    ref = go()
    assert own.get_status() == 0
    own.set_wait_limit(0)
    out = go()
    assert own.get_status() & native.TQ_DEVERR_TIMEOUT
    assert bool(torch.isfinite(out.float()).all())
    own.set_wait_limit(native.TQ_DEFAULT_WAIT_LIMIT)
    assert torch.equal(go(), ref) and own.get_status() == 0


def test_what_a_workspace_held_does_not_matter():
    for c in (case(512, 16, 4, [9000, 20], seed=8), case(256, 16, 4, [5000, 300], Tq=30, seed=8)):
        ref = run(c)
        ws = codec().workspace_latent(2, 1 if c["q"].dim() == 3 else 30, 4, c["dl"])
        for fill in (0xFF, 0x7F, 0):
            ws.fill_(fill)
            assert torch.equal(run(c, workspace=ws), ref)


def test_two_graphs_with_a_workspace_each_and_another_stream():
    c, p = case(512, 16, 4, [5000, 200], seed=8), case(512, 16, 4, [5000, 200], Tq=30, seed=8)
    rd, rp = run(c), run(p)
    k = codec()
    wd, wp = k.workspace_latent(2, 1, 4, 512), k.workspace_latent(2, 30, 4, 512)
    od, op = torch.zeros_like(rd), torch.zeros_like(rp)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    sm = scale(c)
    with torch.cuda.graph(g1):
        k.decode_attention_latent(c["q"], c["pool"], c["table"], c["lens"], 16, c["nb"], sm, workspace=wd, out=od)
    with torch.cuda.graph(g2):
        k.prefill_attention_latent(p["q"], p["pool"], p["table"], p["lens"], 16, p["nb"], sm, workspace=wp, out=op)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s1):
            g1.replay()
        with torch.cuda.stream(s2):
            g2.replay()
    torch.cuda.synchronize()
    assert torch.equal(od, rd) and torch.equal(op, rp)
    out = k.decode_attention_latent(c["q"], c["pool"], c["table"], c["lens"], 16, c["nb"], sm, stream=s1)
    s1.synchronize()
    assert torch.equal(out, rd)
    # lengths changed between replays
    c["lens"].copy_(torch.tensor([130, 4000], dtype=torch.int32).clamp(max=200))
    g1.replay()
    torch.cuda.synchronize()
    ref, bound = reference(c)
    check(od, ref, bound)


def test_two_calls_at_once():
    cases = [case(512, 64, 20, [3000, 70, 511], seed=21), case(256, 32, 100, [900, 1, 2049], seed=22), case(512, 32, 6, [700, 40], Tq=30, seed=23)]
    refs = [run(c) for c in cases]
    spaces = [codec().workspace_latent(len(c["lens"]), 1 if c["q"].dim() == 3 else c["q"].shape[1], c["q"].shape[-2], c["dl"]) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = []
    for _ in range(8):
        for c, w, s in zip(cases, spaces, streams):
            with torch.cuda.stream(s):
                call = codec().decode_attention_latent if c["q"].dim() == 3 else codec().prefill_attention_latent
                outs.append(call(c["q"], c["pool"], c["table"], c["lens"], c["P"], c["nb"], scale(c), workspace=w))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, refs[i % len(cases)])


# ---- append ------------------------------------------------------------------------------------------------

APPEND = [
    (512, 64, 128, 7, True, True),
    (512, 16, 20, 1, False, False),
    (256, 32, 3, 40, True, False),
    (256, 16, 65, 1100, False, True),
    (512, 32, 1, 1500, True, True),
    (512, 64, 0, 33, True, False),
]


@pytest.mark.parametrize("dl,P,Hq,T,normed,interleaved", APPEND)
@pytest.mark.parametrize("rotated", [True, False])
def test_append(dl, P, Hq, T, normed, interleaved, rotated):
    k = codec()
    g = torch.Generator().manual_seed(T + Hq)
    nb = -(-T // P) + 2
    slots = torch.randperm(nb * P, generator=g)[:T]
    slots[torch.arange(T) % 5 == 3] = -1
    live = slots >= 0
    pos = torch.randint(0, 50, (T,), generator=g)
    kv = torch.randn(T, dl + 64 + 16, generator=g).to(torch.bfloat16).to(DEV)
    heads = torch.randn(T, max(Hq, 1), 128 + 64, generator=g).to(torch.bfloat16).to(DEV)
    weight = torch.randn(dl, generator=g).to(torch.bfloat16).to(DEV) if normed else None
    rope = k.rope_table(50, 64)
    was = torch.randn(nb, P, dl + 64, generator=g).to(torch.bfloat16).to(DEV)
    pool = was.clone()
    query = torch.full((T, max(Hq, 1), dl + 64), 7.0, dtype=torch.bfloat16, device=DEV)
    more = dict(positions=pos.to(DEV), rope=rope, interleaved=interleaved) if rotated else {}
    if Hq:
        more.update(q=heads[..., 128:], q_out=query[..., dl:])
    k.append_latent(kv[:, 16: 16 + dl], kv[:, 16 + dl:], slots.to(DEV), pool, P, nb, norm_weight=weight, norm_eps=1e-5, **more)
    torch.cuda.synchronize()
    assert k.get_status() == 0
    turn = (lambda x: R.rotate(x.cpu(), rope.cpu(), pos, interleaved).to(torch.bfloat16)) if rotated else (lambda x: x.cpu())
    flat, old = pool.flatten(0, 1).cpu(), was.flatten(0, 1).cpu()
    rest = torch.ones(nb * P, dtype=torch.bool)
    rest[slots[live]] = False
    assert torch.equal(flat[rest], old[rest])
    got = flat[slots[live]]
    assert torch.equal(got[:, dl:], turn(kv[:, None, 16 + dl:])[live, 0])
    c = kv[:, 16: 16 + dl].cpu()[live]
    if normed:
        y = R.norm(c, weight.cpu(), 1e-5)
        assert bool(((got[:, :dl].double() - y).abs() <= R.norm_bound(y, dl)).all())
    else:
        assert torch.equal(got[:, :dl], c)
    if Hq:
        want = torch.full((T, Hq, dl + 64), 7.0, dtype=torch.bfloat16)
        want[live, :, dl:] = turn(heads[..., 128:])[live]
        assert torch.equal(query.cpu(), want)


def test_append_in_place_and_in_other_layouts():
    k = codec()
    g = torch.Generator().manual_seed(5)
    T, Hq, dl, P = 70, 9, 256, 16
    kv = torch.randn(T, dl + 64, generator=g).to(torch.bfloat16).to(DEV)
    q = torch.randn(Hq, T, 64, generator=g).to(torch.bfloat16).to(DEV)  # heads outermost
    slots, pos, rope = torch.arange(T, device=DEV), torch.arange(T, device=DEV), k.rope_table(T, 64)
    pool = k.alloc_pool_latent(5, P, dl)
    out = k.append_latent(kv[:, :dl], kv[:, dl:], slots, pool, P, 5, q=q.transpose(0, 1), positions=pos, rope=rope)
    same = q.clone().transpose(0, 1)
    assert k.append_latent(kv[:, :dl], kv[:, dl:], slots, pool, P, 5, q=same, q_out=same, positions=pos, rope=rope) is same
    torch.cuda.synchronize()
    assert out.shape == (T, Hq, 64) and torch.equal(out, same) and k.get_status() == 0
    assert torch.equal(out.cpu(), R.rotate(q.transpose(0, 1).cpu(), rope.cpu(), pos.cpu(), False).to(torch.bfloat16))
    one = k.append_latent(kv[:1, :dl], kv[:1, dl:], slots[:1], pool, P, 5, q=q.transpose(0, 1)[:1], positions=pos[:1], rope=rope)
    assert torch.equal(one, out[:1])


def test_append_of_bad_slots_and_positions():
    k = codec()
    pool = k.alloc_pool_latent(2, 16, 256)
    x = torch.ones(4, 320, dtype=torch.bfloat16, device=DEV)
    q = torch.ones(4, 2, 64, dtype=torch.bfloat16, device=DEV)
    rope = k.rope_table(8, 64)
    o = k.append_latent(x[:, :256], x[:, 256:], torch.tensor([3, 32, -5, 9], device=DEV), pool, 16, 2, q=q,
                        positions=torch.tensor([0, 0, 0, 8], device=DEV), rope=rope)
    assert k.get_status() == native.TQ_DEVERR_SLOT_RANGE | native.TQ_DEVERR_POSITION
    rows = pool.flatten(0, 1).abs().sum(1)
    assert float(rows[3]) > 0 and float(rows.sum()) == float(rows[3])
    assert torch.all(o[1:] == 0) and torch.all(o[0] == 1)
    none = torch.empty(0, 320, dtype=torch.bfloat16, device=DEV)
    k.append_latent(none[:, :256], none[:, 256:], torch.empty(0, dtype=torch.int64, device=DEV), pool, 16, 2)
    assert k.get_status() == 0


def test_append_captured():
    k = codec()
    g = torch.Generator().manual_seed(6)
    x = torch.randn(5, 576, generator=g).to(torch.bfloat16).to(DEV)
    pool, other = k.alloc_pool_latent(3, 64, 512), k.alloc_pool_latent(3, 64, 512)
    slots = torch.tensor([0, 64, 65, 100, -1], device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        k.append_latent(x[:, :512], x[:, 512:], slots, pool, 64, 3)
    x.mul_(2)
    graph.replay()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    k.append_latent(x[:, :512], x[:, 512:], slots, other, 64, 3, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(pool, other) and torch.equal(pool[1, 1], x[2])


# ---- refusals, and the set as it is used ---------------------------------------------------------------------

def test_refusals():
    c = case(512, 16, 4, [40], seed=9)
    k = codec()
    ws = k.workspace_latent(1, 1, 4, 512)
    ok = (k.handle, c["q"].data_ptr(), c["pool"].data_ptr(), c["table"].data_ptr(), c["lens"].data_ptr())
    out = torch.empty(1, 4, 512, dtype=torch.bfloat16, device=DEV)

    def refused(status, word, B=1, tq=None, Hq=4, dl=512, P=16, maxb=c["table"].shape[1], nb=c["nb"], sm=0.1, w=ws.data_ptr(),
                n=ws.numel(), o=out.data_ptr(), first=ok):
        with pytest.raises(native.TQError) as e:
            if tq is None:
                native.tq_decode_attention_latent(*first, B, Hq, dl, P, maxb, nb, sm, w, n, o, 0)
            else:
                native.tq_prefill_attention_latent(*first, B, tq, Hq, dl, P, maxb, nb, sm, w, n, o, 0)
        assert e.value.status == status and word in str(e.value), str(e.value)

    for tq in (None, 1):
        refused(native.TQ_ERR_UNSUPPORTED, "page_size", P=128, tq=tq)
        refused(native.TQ_ERR_UNSUPPORTED, "latent_dim", dl=384, tq=tq)
        refused(native.TQ_ERR_INVALID_ARG, "bad sizes", B=-1, tq=tq)
        refused(native.TQ_ERR_INVALID_ARG, "bad sizes", Hq=0, tq=tq)
        refused(native.TQ_ERR_INVALID_ARG, "bad sizes", maxb=0, tq=tq)
        refused(native.TQ_ERR_INVALID_ARG, "sm_scale", sm=float("inf"), tq=tq)
        refused(native.TQ_ERR_INVALID_ARG, "workspace", n=ws.numel() - 1, tq=tq)
        refused(native.TQ_ERR_INVALID_ARG, "workspace", w=0, tq=tq)
        refused(native.TQ_ERR_UNSUPPORTED, "positions", maxb=1 << 28, tq=tq)
        refused(native.TQ_ERR_UNSUPPORTED, "too large", nb=1 << 40, tq=tq)
        refused(native.TQ_ERR_INVALID_ARG, "NULL", o=0, tq=tq)
        refused(native.TQ_ERR_INVALID_ARG, "misaligned", o=out.data_ptr() + 2, tq=tq)
    refused(native.TQ_ERR_INVALID_ARG, "bad sizes", tq=0)
    refused(native.TQ_ERR_UNSUPPORTED, "too many", B=1 << 20, tq=1 << 12)
    for bad in (dict(block_table=c["table"].long()), dict(q=c["q"].float()), dict(q=c["q"].cpu()), dict(pool=c["pool"][:, :8]),
                dict(seq_lens=c["lens"].long()), dict(workspace=torch.empty(1 << 26, dtype=torch.uint8, device=DEV)[::2]),
                dict(out=out[:, :2]), dict(q=c["q"][0])):
        a = dict(q=c["q"], pool=c["pool"], block_table=c["table"], seq_lens=c["lens"])
        a.update(bad)
        with pytest.raises(ValueError):
            k.decode_attention_latent(page_size=16, num_blocks=c["nb"], sm_scale=0.1, **a)


def test_append_refusals():
    k = codec()
    x = torch.zeros(4, 320, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device=DEV)
    pool, slots = k.alloc_pool_latent(2, 16, 256), torch.zeros(4, dtype=torch.int64, device=DEV)

    def refused(status, word, lat=x.data_ptr(), T=4, dl=256, Hq=2, ls=320, ks=320, qs=128, qh=64, eps=0.0, w=0, pos=0, rope=0, rows=0,
                style=0, P=16, nb=2, qq=q.data_ptr(), o=q.data_ptr(), os=128, oh=64, p=pool.data_ptr()):
        with pytest.raises(native.TQError) as e:
            native.tq_append_latent(k.handle, lat, x.data_ptr() + 512, qq, T, dl, Hq, ls, ks, qs, qh, w, eps, pos, rope, rows, style,
                                    slots.data_ptr(), p, P, nb, o, os, oh, 0)
        assert e.value.status == status and word in str(e.value), str(e.value)

    I, U = native.TQ_ERR_INVALID_ARG, native.TQ_ERR_UNSUPPORTED
    for kw in (dict(dl=128), dict(P=8), dict(style=2), dict(T=1 << 31), dict(nb=1 << 40)):
        refused(U, "tq_append_latent", **kw)
    for kw in (dict(T=-1), dict(Hq=0), dict(nb=0), dict(qq=0), dict(o=0), dict(lat=0), dict(p=0), dict(rope=x.data_ptr()),
               dict(rope=x.data_ptr(), pos=slots.data_ptr()), dict(lat=x.data_ptr() + 2), dict(ls=248), dict(ls=324), dict(ks=56), dict(qs=56),
               dict(qh=0), dict(os=4), dict(oh=-64), dict(w=x.data_ptr(), eps=-1.0), dict(w=x.data_ptr(), eps=float("nan"))):
        refused(I, "tq_append_latent", **kw)


def test_append_into_rows_that_overlap_is_refused():
    k = codec()
    T, Hq = 5, 3
    x, q = torch.randn(T, 320, device=DEV).bfloat16(), torch.randn(T, Hq, 64, device=DEV).bfloat16()
    pool, slots = k.alloc_pool_latent(1, 16, 256), torch.arange(T, device=DEV)
    room = torch.zeros(T * Hq * 64, dtype=torch.bfloat16, device=DEV)
    for st, sh, ok in ((64, 64, False), (64 * Hq - 8, 64, False), (64, 64 * T - 8, False), (64 * Hq, 64, True), (64, 64 * T, True)):
        out = torch.as_strided(room, (T, Hq, 64), (st, sh, 1))
        if ok:
            k.append_latent(x[:, :256], x[:, 256:], slots, pool, 16, 1, q=q, q_out=out)
            assert torch.equal(out, q)
        else:
            with pytest.raises(native.TQError, match="overlap"):
                k.append_latent(x[:, :256], x[:, 256:], slots, pool, 16, 1, q=q, q_out=out)


@pytest.mark.parametrize("dl,P,Hq", [(512, 64, 20), (256, 16, 5)])
def test_a_prompt_and_some_tokens_end_to_end(dl, P, Hq):
    """The set as it is used: append a prompt's chunks and attend to them, then token by token."""
    k = codec()
    nb, D = 12, dl + 64
    g = torch.Generator().manual_seed(10)
    table = torch.stack([torch.arange(0, 6), torch.arange(6, 12)]).to(torch.int32)
    rope = k.rope_table(6 * P, 64)
    pool = k.alloc_pool_latent(nb, P, dl)
    weight = torch.randn(dl, generator=g).to(torch.bfloat16).to(DEV)
    ws = k.workspace_latent(2, 37, Hq, dl)
    rows = [torch.empty(0, D, dtype=torch.bfloat16) for _ in range(2)]
    lens = [0, 0]
    for new in (37, 20, 1, 1, 2, 1):
        pos = torch.cat([torch.arange(a, a + new) for a in lens])
        seq = torch.arange(2).repeat_interleave(new)
        slots = (table[seq, pos // P].long() * P + pos % P).to(DEV)
        kv = torch.randn(2 * new, D, generator=g).to(torch.bfloat16).to(DEV)
        query = torch.randn(2 * new, Hq, D, generator=g).to(torch.bfloat16).to(DEV)
        part = query[..., dl:]
        turned = R.rotate(part.cpu(), rope.cpu(), pos, True).to(torch.bfloat16)
        k.append_latent(kv[:, :dl], kv[:, dl:], slots, pool, P, nb, q=part, q_out=part, positions=pos.to(DEV), rope=rope,
                        interleaved=True, norm_weight=weight)
        assert torch.equal(query[..., dl:].cpu(), turned)
        y = R.norm(kv[:, :dl].cpu(), weight.cpu(), 1e-6)
        held = pool.flatten(0, 1)[slots].cpu()
        assert bool(((held[:, :dl].double() - y).abs() <= R.norm_bound(y, dl)).all())
        assert torch.equal(held[:, dl:], R.rotate(kv[:, None, dl:].cpu(), rope.cpu(), pos, True).to(torch.bfloat16)[:, 0])
        lens = [a + new for a in lens]
        c = dict(q=query.view(2, new, Hq, D) if new > 1 else query, pool=pool, table=table.to(DEV),
                 lens=torch.tensor(lens, dtype=torch.int32, device=DEV), nb=nb, P=P, dl=dl)
        ref, bound = reference(c)
        check(run(c, workspace=ws), ref, bound)
    assert k.get_status() == 0
