"""Appends at the edges of their contract."""
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


def pools_with_something(codec, nb, H, P, seed):
    g = torch.Generator().manual_seed(seed)
    pools = codec.alloc_pools_fp8(nb, H, P)
    for p, s in zip(pools[:2], pools[2:]):
        c = torch.randint(1, 127, p.shape, generator=g) | (torch.randint(0, 2, p.shape, generator=g) << 7)
        p.view(torch.uint8).copy_(c.to(torch.uint8))
        s.copy_(2.0 ** torch.randint(-11, -6, s.shape, generator=g).float())
    return pools


def state(pools):
    return [p.view(torch.uint8).cpu().numpy().copy() for p in pools[:2]] + [s.cpu().numpy().copy() for s in pools[2:]]


@pytest.mark.parametrize("d,P,H", [(128, 16, 2), (128, 32, 5), (256, 16, 1), (256, 32, 3)])
@pytest.mark.parametrize("T", [1, 5, 1100])   # few tokens, and many (another cut into blocks)
@pytest.mark.parametrize("row", [0, 3])
def test_a_run_without_a_written_token_changes_nothing(d, P, H, T, row):
    """Every position of some runs lies outside the table, of others only some, of the rest none."""
    codec = _codec(d)
    g = torch.Generator().manual_seed(T + row)
    rope = codec.rope_table(40, d)
    lens, total = [], 0
    while total < T:
        lens.append(min(1 + (7 * len(lens)) % (P - row), T - total))
        total += lens[-1]
    nb = len(lens) + 1
    perm = torch.randperm(nb, generator=g)
    slots = torch.cat([perm[i] * P + row + torch.arange(n) for i, n in enumerate(lens)])
    pos = torch.randint(0, 40, (T,), generator=g)
    ok = np.ones(T, bool)
    at = 0
    for i, n in enumerate(lens):
        if i % 3 != 1:  # of every three runs: none written, all written, all but the last of the run written
            bad = torch.arange(at, at + n) if i % 3 == 0 else torch.tensor([at + n - 1])
            pos[bad] = torch.where(bad % 2 == 0, torch.tensor(40), torch.tensor(-1))
            ok[bad.numpy()] = False
        at += n
    x = (torch.randn(T, H, d, generator=g) * 3).to(torch.bfloat16)
    k, v = x.to(DEV), (0.5 * x).to(torch.bfloat16).to(DEV)
    pools = pools_with_something(codec, nb, H, P, seed=T)
    # an old scale below the least that a page may ask for is no reason to change it either
    pools[2][perm[0]] = 2.0 ** -110
    want = state(pools)
    table = rope.cpu().numpy()
    rk = np.stack([R.rotate(R.bf16(k[t:t + 1])[0], int(pos[t]) if ok[t] else 0, table, False) for t in range(T)])
    live = np.zeros(T, bool)  # tokens of runs that have a written one
    at = 0
    for n in lens:
        live[at: at + n] = ok[at: at + n].any()
        at += n
    masked = np.where(live, slots.numpy(), -1)
    kc, vc, ks, vs = want
    ks64, vs64 = ks.astype(np.float64), vs.astype(np.float64)
    R.append_fp8(kc, ks64, rk, masked, ok, P)
    R.append_fp8(vc, vs64, R.bf16(v), masked, ok, P)
    codec.append_kv_fp8(k, v, slots.to(DEV), *pools, P, nb, positions=pos.to(DEV), rope=rope)
    torch.cuda.synchronize()
    assert codec.get_status() == native.TQ_DEVERR_POSITION
    got = state(pools)
    assert np.array_equal(got[2], ks64) and np.array_equal(got[3], vs64)
    assert np.array_equal(got[0], kc) and np.array_equal(got[1], vc)


@pytest.mark.parametrize("d,P,H", [(128, 16, 2), (128, 32, 1), (256, 16, 3), (256, 32, 1)])
@pytest.mark.parametrize("zero", [0.0, -0.0])
def test_a_zero_scale_on_a_continued_page(d, P, H, zero):
    """Rows under a zero scale stand for zeros, and still do when new rows give the page its scale."""
    codec = _codec(d)
    g = torch.Generator().manual_seed(d + P)
    pools = pools_with_something(codec, 3, H, P, seed=1)
    for s in pools[2:]:
        s[1] = zero
    want = state(pools)
    x = torch.randn(3, H, d, generator=g).to(torch.bfloat16)
    slots = torch.tensor([P + 5, P + 6, 2 * P + 1])
    for c, s in ((want[0], 2), (want[1], 3)):
        sc = want[s].astype(np.float64)
        R.append_fp8(c, sc, R.bf16(x), slots.numpy(), np.ones(3, bool), P)
        want[s] = sc
    assert np.all((want[0][1, :, :5] & 127) == 0)
    codec.append_kv_fp8(x.to(DEV), x.to(DEV), slots.to(DEV), *pools, P, 3)
    torch.cuda.synchronize()
    assert codec.get_status() == 0
    got = state(pools)
    for a, b in zip(got, want):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("d,Hq,r,interleaved,T", [(128, 8, 128, False, 700), (128, 5, 64, True, 2000), (256, 3, 80, False, 33),
                                                  (256, 7, 256, True, 1500), (128, 2, 0, False, 40), (128, 6, 32, True, 1)])
def test_queries_in_place(kind, d, Hq, r, interleaved, T):
    """q_out = q gives what another q_out gets; rows of skipped tokens stay."""
    P, H = 16, 2
    codec = _codec(d)
    g = torch.Generator().manual_seed(T)
    nb = -(-T // P) + 1
    q = torch.randn(T, Hq, d, generator=g).to(torch.bfloat16).to(DEV)
    k, v = [torch.randn(T, H, d, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2)]
    slots = torch.arange(T).to(DEV)
    if T > 20:
        slots[T - 1] = -1
    more = dict(positions=torch.randint(0, 30, (T,), generator=g).to(DEV), rope=codec.rope_table(30, r), interleaved=interleaved) \
        if r else {}
    call, pools = (codec.append_kv_bf16, codec.alloc_pools_bf16(nb, H, P)) if kind == "bf16" else \
        (codec.append_kv_fp8, codec.alloc_pools_fp8(nb, H, P))
    apart = q.clone()
    call(k, v, slots, *pools, P, nb, q=q, q_out=apart, **more)
    same = q.clone()
    assert call(k, v, slots, *pools, P, nb, q=same, q_out=same, **more) is same
    torch.cuda.synchronize()
    assert torch.equal(apart, same) and codec.get_status() == 0
    assert T <= 20 or torch.equal(same[T - 1], q[T - 1])
    if r == d:
        assert not torch.equal(same, q)
