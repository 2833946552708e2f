"""Latent pages at the ends of their ranges, on both of the attention's kernels."""
import ctypes

import pytest
import torch

import latent as R
from rotated_codebook_kv_gb300 import Codec, native
from test_gpu_latent import DEV, case, check, codec, reference, run

pytestmark = pytest.mark.gpu

# the kernel of up to 64 rows a sequence and that of more, one query token and several
SHAPES = [(512, 4, None), (256, 4, None), (512, 100, None), (256, 100, None), (512, 4, 5), (256, 30, 7)]


@pytest.mark.parametrize("dl,Tq", [(512, 64), (256, 64), (512, 128), (256, 128)])
def test_the_join_waits_no_longer_than_the_wait_limit(dl, Tq):
    """A long sequence cut into many pieces; a NaN in its last token keeps the worker of the last piece for some 50 to 200 us
    (it looks for the rows that see it), while the others wait for it to join them: longer than a limit of 30 us, which the
    barriers of a tile stay below."""
    own = Codec(128, 4, 4, 64)
    n = 20000
    c = case(dl, 16, 1, [n], Tq=Tq, seed=31)
    c["pool"][int(c["table"][0, (n - 1) // 16]), (n - 1) % 16, 3] = float("nan")
    ws = own.workspace_latent(1, Tq, 1, dl)

    def go():
        out = torch.full((1, Tq, 1, dl), 777.0, dtype=torch.bfloat16, device=DEV)
        own.prefill_attention_latent(c["q"], c["pool"], c["table"], c["lens"], 16, c["nb"], 0.07, workspace=ws, out=out)
        torch.cuda.synchronize()
        return out[0, :, 0]

    ref = go()
    assert own.get_status() == 0
    assert bool(torch.isfinite(ref[:-1].float()).all()) and bool(torch.isnan(ref[-1]).all())
    own.set_wait_limit(60000)
    for _ in range(3):
        out = go()
        assert own.get_status() == native.TQ_DEVERR_TIMEOUT
        # whoever gave up has written zeros in its part of the rows, and nothing is left as it was
        parts, want = out.view(Tq, -1, 256), ref.view(Tq, -1, 256)
        right = ((parts == want) | (torch.isnan(want) & torch.isnan(parts))).all(-1)
        zero = (parts == 0).all(-1)
        assert bool((right | zero).all()) and bool(zero.any())
    own.set_wait_limit(native.TQ_DEFAULT_WAIT_LIMIT)
    assert torch.equal(go()[:-1], ref[:-1]) and own.get_status() == 0


def rising(c, rise, first):
    """Scores (in powers of two) of 0 for the first tokens and of `rise` from token `first` on, latents near bf16's largest."""
    dl, P = c["dl"], c["P"]
    c["q"].zero_()
    c["q"][..., dl] = 1
    g = torch.Generator(device=DEV).manual_seed(1)
    for b, n in enumerate(c["lens"].tolist()):
        for i, blk in enumerate(c["table"][b].tolist()):
            m = min(P, n - i * P)
            if m <= 0:
                break
            c["pool"][blk, :m, :dl] = torch.where(torch.rand(m, dl, device=DEV, generator=g) < 0.5, 2.9e38, 3.0e38).to(torch.bfloat16)
            c["pool"][blk, :m, dl:] = 0
            t = torch.arange(i * P, i * P + m, device=DEV)
            c["pool"][blk, :m, dl] = torch.where(t < first, 0.0, rise).to(torch.bfloat16)
    return c


@pytest.mark.parametrize("rise", [7.5, 15.875, 16.5, 31.75, 40.0])
@pytest.mark.parametrize("dl,Hq,Tq", SHAPES)
def test_values_near_the_largest_under_rising_scores(dl, Hq, Tq, rise):
    """Later scores above the first ones: sums of probabilities times values stay finite before the division."""
    c = rising(case(dl, 16, Hq, [700, 9000], Tq=Tq, seed=7), rise, 130)
    sm = 0.6931471805599453  # a score is a power of two
    ref, bound = reference(c, sm)
    check(run(c, sm), ref, bound)


def onehot(c, q, lo):
    """Queries of one coordinate each, of size q and both signs; latents from size lo on, so that scores are single products."""
    dl = c["dl"]
    g = torch.Generator(device=DEV).manual_seed(2)
    flat = c["q"].view(-1, dl + 64)
    flat.zero_()
    j = torch.randint(0, dl + 64, (flat.shape[0],), generator=g, device=DEV)
    s = torch.randint(0, 2, (flat.shape[0],), generator=g, device=DEV) * 2.0 - 1
    flat[torch.arange(flat.shape[0], device=DEV), j] = (s * q).to(torch.bfloat16)
    x = torch.randn(c["pool"].shape, device=DEV, generator=g)
    c["pool"].copy_(torch.where(torch.isfinite(c["pool"]), x * lo, c["pool"].float()))
    return c


@pytest.mark.parametrize("sm", [0.07, -0.07])
@pytest.mark.parametrize("power", [22, 26, 30, 33, 40, 80])
@pytest.mark.parametrize("dl,Hq,Tq", SHAPES)
def test_scores_of_any_size(dl, Hq, Tq, power, sm):
    """Scores of up to 2^82 times the scale, each a single product: the token with the largest takes all, ties share."""
    c = onehot(case(dl, 16, Hq, [40, 700, 5000], Tq=Tq, seed=9), 2.0 ** (power // 2), 2.0 ** (power - power // 2))
    out = run(c, sm).double()
    q4 = c["q"].view(3, -1, Hq, dl + 64).double()
    o4 = out.view(3, -1, Hq, dl)
    tq = q4.shape[1]
    for b, L in enumerate(c["lens"].tolist()):
        k = c["pool"][c["table"][b, : -(-L // 16)].long()].double().flatten(0, 1)[:L]
        for i in range(tq):
            n = L - tq + 1 + i
            x = (q4[b, i] @ k[:n].T) * sm
            w = torch.softmax(x, -1)
            top2 = x.topk(2, -1).values
            sure = (top2[:, 0] - top2[:, 1] > 64) | (top2[:, 0] == top2[:, 1])  # what is between 0 and 64 keeps some weight
            ref = w @ k[:n, :dl]
            assert int(sure.sum()) > 0
            tol = 2.0 ** -8 * ref.abs() + 2.0 ** -20 * k[:n, :dl].abs().amax(0)
            assert bool(((o4[b, i] - ref).abs() <= tol)[sure].all())
    assert bool(torch.isfinite(out).all()) and codec().get_status() == 0


@pytest.mark.parametrize("dl,Hq,Tq", SHAPES)
def test_tokens_of_an_infinite_negative_score_across_pieces(dl, Hq, Tq):
    """An infinite coordinate whose score is -inf has no weight, and the coordinate itself is 0 times infinity, however the
    sequence is cut."""
    n, j = 6000, 9
    for first in (0, 64, 128, 192, 256, 320, 384, 448, 512, 640, 768, 1024, 5990):
        c = case(dl, 16, Hq, [n], Tq=Tq, seed=15)
        c["q"][..., j] = c["q"][..., j].abs() + 0.5
        ok = torch.ones(1, n, dtype=torch.bool, device=DEV)
        ok[0, first:] = False
        ref, bound = reference(c, ok=ok)
        t = torch.arange(first, n, device=DEV)
        c["pool"][c["table"][0, t // 16].long(), t % 16, j] = float("-inf")
        out = run(c)
        seen = out if Tq is None else out[:, max(0, Tq - (n - first)):]
        assert bool(torch.isnan(seen[..., j]).all()), first
        rest = torch.arange(dl, device=DEV) != j
        check(out[..., rest], ref[..., rest], bound[..., rest])


def refused(status, word, T=4, Hq=2, ls=320, ks=320, qs=128, qh=64, q=1 << 20, o=1 << 21, os=128, oh=64):
    """An append that is refused before anything is launched; its pointers lead nowhere."""
    at = 1 << 22
    with pytest.raises(native.TQError, match=word) as e:
        native.tq_append_latent(codec().handle, at, at, q, T, 256, Hq, ls, ks, qs, qh, 0, 0.0, 0, 0, 0, 0, at, at, 16, 2, o, os, oh, 0)
    assert e.value.status == status


@pytest.mark.parametrize("T,stride", [((1 << 29) + 1, 1 << 35), ((1 << 29) + 1, 1 << 34), ((1 << 30) - 1, 1 << 40), ((1 << 20) + 1, 1 << 40)])
@pytest.mark.parametrize("which", ["ls", "ks", "qs", "os"])
def test_append_of_rows_whose_offsets_pass_64_bits_is_refused(T, stride, which):
    refused(native.TQ_ERR_UNSUPPORTED, "too far apart", T=T, **{which: stride})


def test_outputs_over_the_queries_with_other_strides_are_refused():
    k = codec()
    T, Hq = 6, 4
    x, pool, slots = torch.randn(T, 320, device=DEV).bfloat16(), k.alloc_pool_latent(1, 16, 256), torch.arange(T, device=DEV)
    room = torch.randn(2 * T * Hq * 64, device=DEV).bfloat16()
    q = room[: T * Hq * 64].view(T, Hq, 64)

    def call(q, q_out):
        return k.append_latent(x[: q.shape[0], :256], x[: q.shape[0], 256:], slots[: q.shape[0]], pool, 16, 1, q=q, q_out=q_out)

    for st, sh in ((64, 64 * T), (64 * Hq * 2, 64), (64 * Hq + 8, 64)):
        with pytest.raises(native.TQError, match="strides"):
            call(q, torch.as_strided(room, (T, Hq, 64), (st, sh, 1)))
    for a, b in ((q[:1], torch.as_strided(room, (1, Hq, 64), (64 * 99, 64, 1))), (q[:, :1], torch.as_strided(room, (T, 1, 64), (64 * Hq, 64 * 99, 1))), (q, q)):
        want = a.clone()
        assert torch.equal(call(a, b), want)


@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("power", [-120, -100, -70, -40, 58, 64, 100, 124])
@pytest.mark.parametrize("dl", [256, 512])
def test_norm_of_latents_of_any_size(dl, power, eps):
    k = codec()
    g = torch.Generator().manual_seed(dl)
    x = (torch.randn(9, dl, generator=g).clamp(-4, 4) * 2.0 ** power).to(torch.bfloat16)
    x[3] = 0
    x[3, 7] = 2.0 ** power
    w = (torch.randn(dl, generator=g).abs() + 0.5).to(torch.bfloat16)
    key = torch.zeros(9, 64, dtype=torch.bfloat16, device=DEV)
    pool = k.alloc_pool_latent(1, 16, dl)
    k.append_latent(x.to(DEV), key, torch.arange(9, device=DEV), pool, 16, 1, norm_weight=w.to(DEV), norm_eps=eps)
    y = R.norm(x, w, eps if eps == 0 else float(torch.tensor(eps, dtype=torch.float32)))
    got = pool[0, :9, :dl].cpu().double()
    assert bool(((got - y).abs() <= R.norm_bound(y, dl)).all())


@pytest.mark.parametrize("Hq", [4, 100])
def test_a_launch_that_fails_fails_alone(Hq):
    """A launch into a capture that has become invalid is refused by the runtime; the next call does not report it again."""
    c = case(512, 16, Hq, [100], seed=1)
    ref = run(c)
    k = codec()
    ws, out = k.workspace_latent(1, 1, Hq, 512), torch.zeros_like(ref)
    x, slots, pool = torch.randn(3, 576, device=DEV).bfloat16(), torch.arange(3, device=DEV), k.alloc_pool_latent(1, 16, 512)
    cuda, s = ctypes.CDLL("libcuda.so.1"), torch.cuda.Stream()
    at = ctypes.c_void_p(s.cuda_stream)
    torch.cuda.synchronize()
    assert cuda.cuStreamBeginCapture_v2(at, 2) == 0  # relaxed
    assert cuda.cuStreamSynchronize(at) != 0         # not allowed: the capture is invalid from here on
    with pytest.raises(native.TQError) as e:
        native.tq_decode_attention_latent(k.handle, c["q"].data_ptr(), c["pool"].data_ptr(), c["table"].data_ptr(), c["lens"].data_ptr(), 1, Hq,
                                          512, 16, c["table"].shape[1], c["nb"], 0.07, ws.data_ptr(), ws.numel(), out.data_ptr(), s.cuda_stream)
    assert e.value.status == native.TQ_ERR_CUDA
    graph = ctypes.c_void_p()
    assert cuda.cuStreamEndCapture(at, ctypes.byref(graph)) != 0 and not graph.value
    k.append_latent(x[:, :512], x[:, 512:], slots, pool, 16, 1)
    torch.cuda.synchronize()
    assert torch.equal(pool[0, :3], x) and torch.equal(run(c), ref) and torch.all(out == 0)


@pytest.fixture
def limited_stream():
    """A stream of a context that may use some 16 SMs."""
    cuda = ctypes.CDLL("libcuda.so.1")
    torch.zeros(1, device=DEV)
    SM, everything, part, rest = 1, *(ctypes.create_string_buffer(512) for _ in range(3))
    count, desc, ctx, stream = ctypes.c_uint(1), ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
    for call in (lambda: cuda.cuDeviceGetDevResource(0, everything, SM),
                 lambda: cuda.cuDevSmResourceSplitByCount(part, ctypes.byref(count), everything, rest, 0, 16),
                 lambda: cuda.cuDevResourceGenerateDesc(ctypes.byref(desc), part, 1),
                 lambda: cuda.cuGreenCtxCreate(ctypes.byref(ctx), desc, 0, 1),
                 lambda: cuda.cuGreenCtxStreamCreate(ctypes.byref(stream), ctx, 1, 0)):
        if call() != 0:
            pytest.skip("no contexts of some of the SMs here")
    yield stream.value
    torch.cuda.synchronize()
    assert cuda.cuStreamDestroy_v2(stream) == 0 and cuda.cuGreenCtxDestroy(ctx) == 0


@pytest.mark.parametrize("dl,Hq,Tq", SHAPES)
def test_on_some_of_the_sms(limited_stream, dl, Hq, Tq):
    for lens in ([9], [3000, 1, 0, 777], [100] * 40):
        c = case(dl, 16, Hq, lens, Tq=Tq, seed=3)
        ref, bound = reference(c)
        whole = run(c)
        ws, out = codec().workspace_latent(len(lens), Tq or 1, Hq, dl), torch.full_like(whole, 7.0)
        torch.cuda.synchronize()
        for _ in range(3):
            run(c, workspace=ws, out=out, stream=limited_stream)
        check(out, ref, bound)
    assert codec().get_status() == 0


@pytest.mark.parametrize("Tq", [None, 2])
def test_a_scale_that_leaves_fp32_in_powers_of_two_is_refused(Tq):
    c = case(256, 16, 2, [40], Tq=Tq, seed=1)
    for sm in (2.4e38, -3.0e38):
        with pytest.raises(native.TQError, match="sm_scale") as e:
            run(c, sm)
        assert e.value.status == native.TQ_ERR_UNSUPPORTED
    c["q"].mul_(1e-38)
    ref, bound = reference(c, 2.3e38)
    check(run(c, 2.3e38), ref, bound)
