"""Attention over 8-bit pages where one strong token with small values stands before a long weak tail; queries and value
scales at the ends of their ranges.

The tail carries most of the output, each of its tokens a probability far below the largest one.  The bound
(`reference`) has no term in which the largest probability of the whole sequence is multiplied by the number of tokens
at the precision of the formats alone.
"""
import numpy as np
import pytest
import torch

import paged8 as R
from rotated_codebook_kv_gb300 import Codec

pytestmark = pytest.mark.gpu
DEV = "cuda"
_codecs = {}


def _codec(d):
    if d not in _codecs:
        _codecs[d] = Codec(d, 4, 4, 64)
    return _codecs[d]


def case(d, P, G, L, Tq, gap, seed=0, strong_value=0.0, at=0):
    """One sequence and kv head: token `at` scores about `gap` nats above a tail with scores of deviation 1; its values
    are strong_value, the others' 1 +- 0.25."""
    g = torch.Generator().manual_seed(seed)
    npg = -(-L // P)
    q = torch.randn((1, G, d) if Tq is None else (1, Tq, G, d), generator=g).to(torch.bfloat16)
    rows = R.bf16(q).reshape(-1, d)
    k = torch.randn(npg * P, d, generator=g)
    # the row whose product with every query is gap sqrt(d)
    k[at] = torch.from_numpy(np.linalg.pinv(rows) @ np.full(len(rows), gap * d ** 0.5)).float()
    v = 1.0 + 0.25 * torch.randn(npg * P, d, generator=g)
    v[at] = strong_value * v[at]
    codes, scales = [], []
    for x in (k, v):
        x = x.view(npg, P, d)
        s = 2.0 ** torch.ceil(torch.log2(x.abs().amax((1, 2)) / 448))
        codes.append((x / s[:, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)[:, None].contiguous())
        scales.append(s[:, None].contiguous())
    return dict(q=q, codes=codes, scales=scales, table=torch.arange(npg, dtype=torch.int32)[None].contiguous(),
                lens=torch.tensor([L], dtype=torch.int32), nb=npg, P=P, d=d, G=G, L=L)


def run(c, splits, sm=None):
    codec = _codec(c["d"])
    call = codec.decode_attention_fp8 if c["q"].dim() == 3 else codec.prefill_attention_fp8
    pools = [x.to(DEV).view(torch.float8_e4m3fn) for x in c["codes"]] + [x.to(DEV) for x in c["scales"]]
    out = call(c["q"].to(DEV), *pools, c["table"].to(DEV), c["lens"].to(DEV), 1, c["P"], c["nb"],
               c["d"] ** -0.5 if sm is None else sm, splits=splits)
    torch.cuda.synchronize()
    assert codec.get_status() == 0
    return out


def reference(c, sm=None):
    """(out, bound) in 64 bits.

    Roundings counted per output element (p the probabilities, v = code vs the values, A = sum p |v|):
      * bf16 output: half a step, 2^-8 |out|;
      * up to eight columns, P as two e4m3 terms of fp16(2^8 p), the largest p vs of a round of 32 tokens at 1: the first
        leaves at most 2^-4 of p, the second 2^-4 of that or half its least step, 2^-10: (2^-8 + 2^-11) p +
        2^-18 max_round(p vs) |code| (1 + 2^-14 for fp16's own least steps);
      * more columns, P in fp16: 2^-11 p, or half the least step, 2^-25, where the largest p vs so far stands at 2^4 or
        above: 2^-29 max(p vs) |code|;
      * scores, exponentials and fp32 sums as in paged8.attention.
    """
    d, P, G, L = c["d"], c["P"], c["G"], c["L"]
    sm = d ** -0.5 if sm is None else sm
    q = R.bf16(c["q"])
    q4 = q.reshape(-1, G, d)
    Tq = len(q4)
    ks, vs = [np.repeat(s[:, 0].double().numpy(), P)[:L] for s in c["scales"]]
    k = R.E4M3[c["codes"][0][:, 0].numpy().reshape(-1, d)[:L]] * ks[:, None]
    ac = np.abs(R.E4M3[c["codes"][1][:, 0].numpy().reshape(-1, d)[:L]])
    v = R.E4M3[c["codes"][1][:, 0].numpy().reshape(-1, d)[:L]] * vs[:, None]
    av, sk = ac * vs[:, None], np.abs(k).sum(1)
    out, bound = np.zeros(q4.shape), np.zeros(q4.shape)
    for i in range(Tq):
        n = L - Tq + 1 + i
        for h in range(G):
            x = (k[:n] @ q4[i, h]) * sm
            w = np.exp(x - x.max())
            p = w / w.sum()
            pv = p * vs[:n]
            o, A = p @ v[:n], p @ av[:n]
            mag = (np.abs(k[:n]) @ np.abs(q4[i, h])) * abs(sm)
            dx = 2.0 ** -17 * np.abs(q4[i, h]).max() * sk[:n] * abs(sm) + d / 16 * 2.0 ** -23 * mag + \
                (np.abs(x) * 1.45 + 8) * 2.0 ** -21
            if Tq * G <= 8:
                top = np.zeros(-(-n // 32) * 32)
                top[:n] = pv
                top = np.repeat(top.reshape(-1, 32).max(1), 32)[:n]
                eps, low = 2.0 ** -8 + 2.0 ** -11, 2.0 ** -18 * (1 + 2.0 ** -14) * top
            else:
                eps, low = 2.0 ** -11, np.full(n, 2.0 ** -29 * pv.max())
            dA = (p * dx) @ av[:n] + (p @ dx) * A
            out[i, h] = o
            bound[i, h] = 2.0 ** -8 * np.abs(o) + eps * A + low @ ac[:n] + dA + (n / 8 + 4) * 2.0 ** -23 * A + 1e-38
    return out.reshape(q.shape), bound.reshape(q.shape)


def check(out, ref, bound):
    got = R.bf16(out)
    assert np.all(np.isfinite(got))
    worst = float((np.abs(got - ref) / bound).max())
    assert worst <= 1.0, f"{worst:.2f} of the bound; largest relative error {np.abs(got / ref - 1).max():.2e}"


@pytest.mark.parametrize("gap", [10.0, 12.0, 13.0, 14.0, 16.0])
@pytest.mark.parametrize("d,P,G,L,Tq", [
    (128, 16, 2, 32768, None),
    (256, 32, 1, 32768, None),
    (128, 32, 2, 20001, 4),      # several query tokens of the decode's kernel
    (256, 16, 1, 20001, 5),
])
def test_decode_keeps_the_tail(d, P, G, L, Tq, gap):
    c = case(d, P, G, L, Tq, gap, seed=int(gap), strong_value=0.02 if gap == 13.0 else 0.0)
    ref, bound = reference(c)
    # the bound is a tight one: the tail's share cannot go missing unseen
    assert float((bound / np.abs(ref)).max()) < 0.06
    for splits in (1, 0):
        check(run(c, splits), ref, bound)


@pytest.mark.parametrize("gap", [11.0, 13.0, 15.0])
@pytest.mark.parametrize("d,P,G,L,Tq", [
    (128, 16, 1, 131072, 9),
    (128, 32, 4, 4096, 3),
    (256, 16, 1, 4096, 9),
    (256, 32, 3, 65536, 4),
])
def test_prefill_keeps_the_tail(d, P, G, L, Tq, gap):
    c = case(d, P, G, L, Tq, gap, seed=int(gap), strong_value=0.02 if gap == 13.0 else 0.0)
    ref, bound = reference(c)
    assert float((bound / np.abs(ref)).max()) < 0.06
    for splits in (1, 0):
        check(run(c, splits), ref, bound)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("Tq", [None, 3, 12])
@pytest.mark.parametrize("at", [5000, 8191 - 40])
def test_strong_token_behind_and_within_the_tail(d, Tq, at):
    """The strong token after the tail (all before it is scaled down) and between two halves of it."""
    c = case(d, 16, 1, 8191, Tq, 14.0, seed=at, at=at)
    ref, bound = reference(c)
    for splits in (1, 3):
        check(run(c, splits), ref, bound)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("Tq", [None, 12])
def test_scores_in_steps_down(d, Tq):
    """Stretches of tokens each 5 nats below the one before: every round's largest far below the running one."""
    L, P = 4096, 16
    c = case(d, P, 1, L, Tq, 0.0, seed=d, strong_value=1.0)
    g = torch.Generator().manual_seed(1)
    u = torch.from_numpy(np.linalg.pinv(R.bf16(c["q"]).reshape(-1, d)) @ np.full(1 if Tq is None else Tq, d ** 0.5)).float()
    lift = 60.0 - 5.0 * (torch.arange(L) // 300)
    k = (0.2 * torch.randn(L, d, generator=g) + lift[:, None] * u).view(L // P, P, d)
    s = 2.0 ** torch.ceil(torch.log2(k.abs().amax((1, 2)) / 448))
    c["codes"][0] = (k / s[:, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)[:, None].contiguous()
    c["scales"][0] = s[:, None].contiguous()
    # the values grow as the probabilities fall, so that every stretch counts
    c["scales"][1] = c["scales"][1] * 2.0 ** torch.round(1.4427 * (60.0 - lift.view(-1, P)[:, :1]))
    ref, bound = reference(c)
    for splits in (1, 0, 4):
        check(run(c, splits), ref, bound)


@pytest.mark.parametrize("d,Tq", [(128, None), (256, None), (128, 3), (128, 20), (256, 20)])
def test_calls_repeat_themselves_bit_for_bit(d, Tq):
    c = case(d, 16, 2, 9000, Tq, 8.0, seed=d)
    for splits in (0, 1, 3):
        first = run(c, splits)
        for _ in range(3):
            assert torch.equal(first, run(c, splits))


@pytest.mark.parametrize("d,Tq", [(128, None), (128, 20), (256, 20)])
def test_long_sequence_of_zero_values(d, Tq):
    """Empty pages (scale 2^-100) among others: denominators neither overflow nor vanish."""
    c = case(d, 16, 1, 70000, Tq, 12.0, seed=3, at=69000)
    c["codes"][1][:] = 0
    c["scales"][1][:] = 2.0 ** -100
    for splits in (1, 0):
        assert torch.all(run(c, splits) == 0)
    c = case(d, 16, 1, 70000, Tq, 20.0, seed=3)  # a strong token of no value, then a few pages that have some
    c["codes"][1][:4300] = 0
    c["scales"][1][:4300] = 2.0 ** -100
    ref, bound = reference(c)
    for splits in (1, 0):
        check(run(c, splits), ref, bound)


@pytest.mark.parametrize("d,Tq", [(128, None), (256, None), (128, 3), (128, 20), (256, 20)])
@pytest.mark.parametrize("big", [120, 122, 125, 127])
def test_largest_queries(d, Tq, big):
    """Queries up to the largest bf16, keys small in the same measure."""
    c = case(d, 16, 1, 300, Tq, 1.0, seed=big, strong_value=1.0)
    q = c["q"].float()
    c["q"] = (q / q.abs().amax() * 1.9921875 * 2.0 ** big).to(torch.bfloat16)
    c["scales"][0] = c["scales"][0] * 2.0 ** (2 - big)
    ref, bound = reference(c)
    for splits in (1, 0):
        check(run(c, splits), ref, bound)


@pytest.mark.parametrize("d,Tq", [(128, None), (256, None), (128, 3), (128, 20), (256, 20)])
@pytest.mark.parametrize("e", [-100, -60, 60, 120])
def test_value_scales_at_the_ends_of_their_range(d, Tq, e):
    c = case(d, 16, 1, 700, Tq, 3.0, seed=5, strong_value=1.0)
    # codes up to 8, so that the largest scale keeps the values finite
    x = c["codes"][1].view(torch.float8_e4m3fn).float() / 64
    c["codes"][1] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    c["scales"][1] = torch.full_like(c["scales"][1], 2.0 ** e)
    ref, bound = reference(c)
    for splits in (1, 2):
        check(run(c, splits), ref, bound)
    c["scales"][1][3:7] = 0.0  # counts as the least
    if e > -100:
        ref, bound = reference(c)
        for splits in (1, 2):
            check(run(c, splits), ref, bound)


@pytest.mark.parametrize("d,G,Tq", [(128, 1, 5), (128, 2, 4), (256, 1, 8), (128, 4, 9), (256, 3, 12)])
@pytest.mark.parametrize("L", [20, 33, 52])
def test_a_later_page_of_far_larger_values_is_not_felt_before_it_is_seen(d, G, Tq, L):
    """Query tokens that see only the pages before one whose value scale is 2^130 larger."""
    c = case(d, 16, G, L, Tq, 1.0, seed=L, strong_value=1.0)
    c["scales"][1][-1] *= 2.0 ** 70
    c["scales"][1][:-1] *= 2.0 ** -60
    ref, bound = reference(c)
    for splits in (1, 2):
        check(run(c, splits), ref, bound)


@pytest.mark.parametrize("d,P,Tq", [(128, 16, None), (256, 16, None), (128, 32, None), (128, 16, 3), (256, 32, 5), (128, 16, 20),
                                    (128, 32, 12), (256, 16, 20)])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_value_scales_of_every_size_side_by_side(d, P, Tq, seed):
    """Every page's value scale somewhere in 2^-85 .. 2^105: all pages have their part of the denominator."""
    c = case(d, P, 1, 700 - 13 * seed, Tq, 2.0, seed=seed, strong_value=1.0)
    g = torch.Generator().manual_seed(seed)
    x = c["codes"][1].view(torch.float8_e4m3fn).float() / 64
    c["codes"][1] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    c["scales"][1] = 2.0 ** torch.randint(-85, 106, c["scales"][1].shape, generator=g).float()
    ref, bound = reference(c)
    for splits in (1, 0, 5):
        check(run(c, splits), ref, bound)
