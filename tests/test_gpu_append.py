"""Appending rotated keys and values to bf16 pages and to 8-bit pages, against plain numpy references.

bf16 pages and rotated queries: the reference rounds the same fp32 products and sums, so the bf16 results agree
bit for bit.  8-bit pages: the fp32 values agree, so scales and codes agree exactly.
"""
import numpy as np
import pytest
import torch

import paged8 as R
from rotated_codebook_kv_gb300 import Codec, native

pytestmark = pytest.mark.gpu
DEV = "cuda"


def to_bf16_bits(x):
    """Nearest-even bf16 bits of fp32-valued x."""
    b = np.asarray(x, np.float32).view(np.uint32)
    return ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)


def make(seed, d, P, Hq, Hkv, past, new, pad=0, r=None, interleaved=False, scale=1.0, strided=True):
    """Packed chunks of sequences with `past` positions in the cache and `new` to append."""
    g = torch.Generator().manual_seed(seed)
    ends = [a + b for a, b in zip(past, new)]
    npg = [-(-e // P) for e in ends]
    nb = sum(npg) + 2
    perm = torch.randperm(nb, generator=g)
    slots, pos, at = [], [], 0
    for a, e, n in zip(past, ends, npg):
        p = torch.arange(a, e)
        slots.append(perm[at: at + n][p // P] * P + p % P)
        pos.append(p)
        at += n
    slots = torch.cat(slots + [torch.full((pad,), -1)]).to(torch.int64)
    pos = torch.cat(pos + [torch.zeros(pad)]).to(torch.int64)
    T = slots.numel()
    if strided:
        qkv = (torch.randn(T, Hq + 2 * Hkv, d, generator=g) * scale).to(torch.bfloat16).to(DEV)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        q, k, v = [(torch.randn(T, h, d, generator=g) * scale).to(torch.bfloat16).to(DEV) for h in (Hq, Hkv, Hkv)]
    r = d if r is None else r
    rope = None
    if r:
        rope = Codec.rope_table(_codec(d), max(ends + [1]), r)
    return dict(q=q, k=k, v=v, slots=slots, pos=pos, nb=nb, rope=rope, interleaved=interleaved, P=P, T=T)


_codecs = {}


def _codec(d):
    if d not in _codecs:
        _codecs[d] = Codec(d, 4, 4, 64)
    return _codecs[d]


def rotated(x, c, positions=True):
    x = R.bf16(x)
    if c["rope"] is None:
        return x
    rope = c["rope"].cpu().numpy()
    return np.stack([R.rotate(x[t], int(c["pos"][t]), rope, c["interleaved"]) for t in range(c["T"])])


def args(c):
    return dict(positions=c["pos"].to(DEV) if c["rope"] is not None else None, rope=c["rope"], interleaved=c["interleaved"])


CASES = [
    # d, P, Hq, Hkv, past, new, pad, rot_dim, interleaved
    (128, 16, 4, 2, [0], [1], 0, None, False),
    (128, 16, 8, 1, [5, 0, 16, 31], [1, 1, 1, 1], 0, None, True),
    (128, 32, 3, 3, [3, 70], [40, 29], 2, 64, False),
    (256, 16, 5, 1, [0, 9], [33, 7], 0, 80, True),
    (256, 32, 16, 2, [1, 64, 40], [95, 3, 200], 1, 256, False),
    (128, 16, 6, 2, [0, 100], [700, 611], 3, 16, False),   # many tokens: 16 to a block
    (256, 32, 2, 1, [7], [1500], 0, 128, True),
    (128, 16, 2, 2, [4], [19], 0, 0, False),               # no rotation
]


@pytest.mark.parametrize("d,P,Hq,Hkv,past,new,pad,r,inter", CASES)
def test_append_bf16(d, P, Hq, Hkv, past, new, pad, r, inter):
    c = make(d + P + Hq, d, P, Hq, Hkv, past, new, pad, r, inter)
    codec = _codec(d)
    kp, vp = [torch.randn(c["nb"], Hkv, P, d).to(torch.bfloat16).to(DEV) for _ in range(2)]
    want_k, want_v = R.bf16_bits(kp).copy(), R.bf16_bits(vp).copy()
    q_out = torch.full((c["T"], Hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
    want_q = R.bf16_bits(q_out).copy()
    got = codec.append_kv_bf16(c["k"], c["v"], c["slots"].to(DEV), kp, vp, P, c["nb"], q=c["q"], q_out=q_out, **args(c))
    torch.cuda.synchronize()
    assert codec.get_status() == 0 and got is q_out
    rq, rk = rotated(c["q"], c), rotated(c["k"], c)
    vb = R.bf16_bits(c["v"])
    for t, s in enumerate(c["slots"].tolist()):
        if s < 0:
            continue
        want_q[t] = to_bf16_bits(rq[t])
        want_k[s // P, :, s % P] = to_bf16_bits(rk[t])
        want_v[s // P, :, s % P] = vb[t]
    assert np.array_equal(R.bf16_bits(q_out), want_q)
    assert np.array_equal(R.bf16_bits(kp), want_k)
    assert np.array_equal(R.bf16_bits(vp), want_v)


def fp8_pools(codec, nb, Hkv, P, seed=0):
    """Pools that hold something: random codes (no NaN) and power-of-two scales."""
    g = torch.Generator().manual_seed(seed)
    d = codec.head_dim
    kp, vp, ks, vs = codec.alloc_pools_fp8(nb, Hkv, P)
    for p, s in ((kp, ks), (vp, vs)):
        c = torch.randint(0, 127, p.shape, generator=g) | (torch.randint(0, 2, p.shape, generator=g) << 7)
        p.view(torch.uint8).copy_(c.to(torch.uint8))
        s.copy_(2.0 ** torch.randint(-11, -6, s.shape, generator=g).float())
    return kp, vp, ks, vs


def codes_of(p):
    return p.view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("d,P,Hq,Hkv,past,new,pad,r,inter", CASES)
def test_append_fp8(d, P, Hq, Hkv, past, new, pad, r, inter):
    c = make(d + P + Hq + 1, d, P, Hq, Hkv, past, new, pad, r, inter)
    codec = _codec(d)
    kp, vp, ks, vs = fp8_pools(codec, c["nb"], Hkv, P, seed=P)
    want = [codes_of(kp).copy(), codes_of(vp).copy(), ks.cpu().double().numpy(), vs.cpu().double().numpy()]
    slots, ok = c["slots"].numpy(), c["slots"].numpy() >= 0
    R.append_fp8(want[0], want[2], rotated(c["k"], c), slots, ok, P)
    R.append_fp8(want[1], want[3], R.bf16(c["v"]), slots, ok, P)
    for again in range(2):  # the same tokens once more change nothing
        q_out = codec.append_kv_fp8(c["k"], c["v"], c["slots"].to(DEV), kp, vp, ks, vs, P, c["nb"], q=c["q"], **args(c))
        torch.cuda.synchronize()
        assert codec.get_status() == 0
        assert np.array_equal(ks.cpu().numpy(), want[2]) and np.array_equal(vs.cpu().numpy(), want[3])
        assert np.array_equal(codes_of(kp), want[0])
        assert np.array_equal(codes_of(vp), want[1])
        if again == 0:
            rq = to_bf16_bits(rotated(c["q"], c))
            rq[slots < 0] = 0
            assert np.array_equal(R.bf16_bits(q_out), rq)


def test_append_without_queries_and_without_tokens():
    codec = _codec(128)
    c = make(3, 128, 16, 2, 2, [0], [20])
    kp, vp, ks, vs = fp8_pools(codec, c["nb"], 2, 16)
    assert codec.append_kv_fp8(c["k"], c["v"], c["slots"].to(DEV), kp, vp, ks, vs, 16, c["nb"], **args(c)) is None
    before = codes_of(kp).copy()
    none = torch.empty(0, 2, 128, dtype=torch.bfloat16, device=DEV)
    no = torch.empty(0, dtype=torch.int64, device=DEV)
    codec.append_kv_fp8(none, none, no, kp, vp, ks, vs, 16, c["nb"])
    codec.append_kv_bf16(none, none, no, *codec.alloc_pools_bf16(3, 2, 16), 16, 3)
    torch.cuda.synchronize()
    assert np.array_equal(codes_of(kp), before) and codec.get_status() == 0


def test_append_one_by_one_equals_at_once_when_scales_do_not_fall_to_subnormals():
    """Power-of-two scales: rows coded anew under a grown scale are the codes that they would have had at once,
    where none becomes subnormal (elements within 2^-6 of the page's largest here)."""
    d, P, H = 128, 16, 2
    codec = _codec(d)
    g = torch.Generator().manual_seed(5)
    T = 16
    mag = 2.0 ** torch.arange(-4, 4, 0.5)[:T].view(T, 1, 1)  # rows grow: the scale grows several times
    x = ((0.9 + 0.1 * torch.rand(T, H, d, generator=g)) * mag).to(torch.bfloat16).to(DEV)
    slots = torch.arange(T).to(DEV)
    one, all_ = [codec.alloc_pools_fp8(1, H, P) for _ in range(2)]
    codec.append_kv_fp8(x, x, slots, *all_, P, 1)
    for t in range(T):
        codec.append_kv_fp8(x[t:t + 1], x[t:t + 1], slots[t:t + 1], *one, P, 1)
    torch.cuda.synchronize()
    for a, b in zip(one, all_):
        assert torch.equal(a.view(torch.uint8) if a.dtype != torch.float32 else a,
                           b.view(torch.uint8) if b.dtype != torch.float32 else b)


def test_append_fp8_extremes():
    """Zeros, the largest bf16, tiny values, infinities and NaN."""
    d, P, H = 128, 16, 1
    codec = _codec(d)
    rows = torch.zeros(6, H, d)
    rows[1] = 3.38e38
    rows[2] = 1e-38
    rows[3, 0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 2.0])
    rows[4] = 448.0
    rows[5] = 449.9
    x = rows.to(torch.bfloat16).to(DEV)
    slots = (torch.arange(6) * P).to(DEV)  # a page each
    kp, vp, ks, vs = codec.alloc_pools_fp8(6, H, P)
    codec.append_kv_fp8(x, x, slots, kp, vp, ks, vs, P, 6)
    torch.cuda.synchronize()
    want = np.zeros((6, H, P, d), np.uint8)
    sc = np.ones((6, H))
    R.append_fp8(want, sc, R.bf16(x), slots.cpu().numpy(), np.ones(6, bool), P)
    assert np.array_equal(codes_of(kp), want) and np.array_equal(ks.cpu().numpy(), sc)
    assert np.array_equal(codes_of(vp), want)
    got = kp[3, 0, 0, :4].float().cpu().numpy() * sc[3, 0]
    assert got[0] == 448 * sc[3, 0] and got[1] == -448 * sc[3, 0] and np.isnan(got[2]) and got[3] == 2.0
    assert sc[0, 0] == 2.0 ** -100 and sc[4, 0] == 1.0 and sc[5, 0] == 2.0


def test_append_bad_slots_positions_and_order():
    d, P, H, nb = 128, 16, 2, 4
    codec = _codec(d)
    g = torch.Generator().manual_seed(11)
    T = 6
    k = torch.randn(T, H, d, generator=g).to(torch.bfloat16).to(DEV)
    rope = codec.rope_table(8, 64)

    def run(slots, pos):
        kp, vp, ks, vs = fp8_pools(codec, nb, H, P, seed=2)
        b = codes_of(kp).copy(), ks.cpu().numpy().copy()
        q_out = torch.full((T, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
        codec.append_kv_fp8(k, k, torch.tensor(slots, device=DEV), kp, vp, ks, vs, P, nb, q=k, q_out=q_out,
                            positions=torch.tensor(pos, device=DEV), rope=rope)
        k16, v16 = codec.alloc_pools_bf16(nb, H, P)
        s8 = codec.get_status()
        codec.append_kv_bf16(k, k, torch.tensor(slots, device=DEV), k16, v16, P, nb, q=k, q_out=q_out.clone(),
                             positions=torch.tensor(pos, device=DEV), rope=rope)
        torch.cuda.synchronize()
        return b, codes_of(kp), ks.cpu().numpy(), q_out, s8, codec.get_status(), k16

    # a slot behind the pool, a negative one, a bad position inside a run
    (b, bs), got, gs, q_out, s8, s16, k16 = run([0, nb * P, -5, 16, 17, 18], [0, 1, 2, 3, 8, 5])
    assert s8 == s16 == native.TQ_DEVERR_SLOT_RANGE | native.TQ_DEVERR_POSITION
    same = got == b
    for s in range(nb * P):
        written = s in (0, 16, 18)
        assert np.all(same[s // P, :, s % P]) == (not written), s
        assert (k16[s // P, :, s % P].abs().max() > 0).item() == written
    for t in range(T):
        assert torch.all(q_out[t] == 7.0).item() == (t in (1, 2, 4))
    # the same page in two places of the call: the later run is left out, whichever it is
    (b, bs), got, gs, _, s8, _, _ = run([0, 1, 16, 2, 3, 17], [0] * 6)
    assert s8 == native.TQ_DEVERR_SLOT_ORDER
    same = got == b
    assert not np.any(np.all(same[0, :, :2], axis=-1)) and np.all(same[0, :, 2:]) and np.all(same[1, :, 1:])
    # the same slot twice
    (b, bs), got, gs, _, s8, _, _ = run([0, 0, 32, 33, 34, 35], [0] * 6)
    assert s8 == native.TQ_DEVERR_SLOT_ORDER


@pytest.mark.parametrize("d,P,H,T", [(128, 16, 2, 1300), (256, 32, 1, 1100), (128, 32, 5, 1024), (256, 16, 3, 999)])
def test_append_many_single_tokens(d, P, H, T):
    """A page per token, in any order; some pages come again within the next 32 tokens, which leaves those out."""
    codec = _codec(d)
    g = torch.Generator().manual_seed(T)
    k, v = [torch.randn(T, H, d, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2)]
    rope = codec.rope_table(50, d)
    pos = torch.randint(0, 50, (T,), generator=g)
    slots = torch.randperm(T, generator=g) * P + torch.randint(0, P - 1, (T,), generator=g)
    for again in (False, True):
        ok = np.ones(T, bool)
        if again:
            # neighbours (the slot itself once more, and an earlier one), one page 15 and one 31 tokens on, around where
            # stretches of 16 and 32 tokens meet
            for a, b, o in ((15, 16, 0), (100, 101, None), (31, 46, 3), (500, 531, 1), (959, 990, 0)):
                slots[b] = slots[a] if o is None else slots[a] // P * P + (slots[a] % P + P - 1 - o) % P
                ok[b] = False
        pools = fp8_pools(codec, T, H, P, seed=T)
        want = [codes_of(pools[0]).copy(), codes_of(pools[1]).copy(), pools[2].cpu().double().numpy(), pools[3].cpu().double().numpy()]
        c = dict(rope=rope, pos=pos, T=T, interleaved=True)
        R.append_fp8(want[0], want[2], rotated(k, c), np.where(ok, slots.numpy(), -1), ok, P)
        R.append_fp8(want[1], want[3], R.bf16(v), np.where(ok, slots.numpy(), -1), ok, P)
        codec.append_kv_fp8(k, v, slots.to(DEV), *pools, P, T, positions=pos.to(DEV), rope=rope, interleaved=True)
        torch.cuda.synchronize()
        assert codec.get_status() == (native.TQ_DEVERR_SLOT_ORDER if again else 0)
        assert np.array_equal(pools[2].cpu().numpy(), want[2]) and np.array_equal(pools[3].cpu().numpy(), want[3])
        assert np.array_equal(codes_of(pools[0]), want[0]) and np.array_equal(codes_of(pools[1]), want[1])


def test_append_captured_in_a_graph_and_on_another_stream():
    d, P = 128, 16
    codec = _codec(d)
    c = make(9, d, P, 4, 2, [3, 30], [50, 1])
    slots, a = c["slots"].to(DEV), args(c)
    ref = fp8_pools(codec, c["nb"], 2, P, seed=1)
    codec.append_kv_fp8(c["k"], c["v"], slots, *ref, P, c["nb"], q=c["q"], **a)
    pools = fp8_pools(codec, c["nb"], 2, P, seed=1)
    q_out = torch.zeros(c["T"], 4, d, dtype=torch.bfloat16, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        codec.append_kv_fp8(c["k"], c["v"], slots, *pools, P, c["nb"], q=c["q"], q_out=q_out, **a)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for x, y in zip(ref, pools):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)) if x.dtype != torch.float32 else torch.equal(x, y)
    other = fp8_pools(codec, c["nb"], 2, P, seed=1)
    s.wait_stream(torch.cuda.current_stream())
    codec.append_kv_fp8(c["k"], c["v"], slots, *other, P, c["nb"], q=c["q"], stream=s, **a)
    s.synchronize()
    assert torch.equal(ref[2], other[2]) and torch.equal(ref[0].view(torch.uint8), other[0].view(torch.uint8))


def test_append_refusals():
    codec = _codec(128)
    P, nb, H = 16, 4, 2
    kp, vp, ks, vs = codec.alloc_pools_fp8(nb, H, P)
    x = torch.zeros(3, H, 128, dtype=torch.bfloat16, device=DEV)
    s = torch.zeros(3, dtype=torch.int64, device=DEV)
    with pytest.raises(native.TQError) as e:  # a rotation that is no multiple of 16
        codec.append_kv_fp8(x, x, s, kp, vp, ks, vs, P, nb, positions=s, rope=torch.zeros(4, 24, device=DEV))
    assert e.value.status == native.TQ_ERR_UNSUPPORTED and "rot_dim" in str(e.value)
    with pytest.raises(native.TQError) as e:
        codec.append_kv_fp8(x, x, s, kp, vp, ks, vs, P, nb, positions=s, rope=torch.zeros(4, 256, device=DEV))
    assert e.value.status == native.TQ_ERR_UNSUPPORTED
    with pytest.raises(native.TQError) as e:
        codec.append_kv_fp8(x, x, s, kp.view(2 * nb, H, 8, 128), vp, ks.repeat(2, 1), vs.repeat(2, 1), 8, 2 * nb)
    assert e.value.status == native.TQ_ERR_UNSUPPORTED and "page_size" in str(e.value)
    wide = torch.zeros(3 * H * 128 + 8, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(native.TQError) as e:  # rows that are not 16-byte aligned
        y = wide[4:4 + 3 * H * 128].view(3, H, 128)
        codec.append_kv_fp8(y, x, s, kp, vp, ks, vs, P, nb)
    assert e.value.status == native.TQ_ERR_INVALID_ARG and "misaligned" in str(e.value)
    with pytest.raises(native.TQError) as e:  # token rows that overlap
        native.tq_append_kv_fp8(codec.handle, 0, x.data_ptr(), x.data_ptr(), 3, 0, H, 0, 128, 256, 0, 0, 0, 0, 0,
                                s.data_ptr(), kp.data_ptr(), vp.data_ptr(), ks.data_ptr(), vs.data_ptr(), P, nb, 0, 0)
    assert e.value.status == native.TQ_ERR_INVALID_ARG and "strides" in str(e.value)


def test_append_refuses_what_no_grid_holds():
    codec = _codec(128)
    x = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device=DEV)
    s = torch.zeros(1, dtype=torch.int64, device=DEV)
    pools = codec.alloc_pools_fp8(1, 2, 16)

    def refused(word, T=1, Hq=2, Hkv=2):
        with pytest.raises(native.TQError) as e:
            native.tq_append_kv_fp8(codec.handle, x.data_ptr(), x.data_ptr(), x.data_ptr(), T, Hq, Hkv, Hq * 128, Hkv * 128,
                                    Hkv * 128, 0, 0, 0, 0, 0, s.data_ptr(), *[p.data_ptr() for p in pools], 16, 1, x.data_ptr(), 0)
        assert e.value.status == native.TQ_ERR_UNSUPPORTED and word in str(e.value), str(e.value)

    refused("too many tokens", T=1 << 30)
    refused("too many tokens", T=1 << 28, Hq=64)
    refused("heads", Hq=(1 << 18) + 1)
    refused("heads", Hkv=(1 << 18) + 1)
