"""Latent pages: refusals that need no GPU, and the reference against plain formulas."""
import types

import pytest
import torch

import latent as R
from rotated_codebook_kv_gb300 import Codec, build, native


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return native.load()


def test_null_handle_refused():
    calls = {
        "tq_append_latent": lambda: native.tq_append_latent(None, 0, 0, 0, 1, 512, 0, 512, 64, 64, 64, 0, 0.0, 0, 0, 0, 0, 0, 0, 16, 1,
                                                            0, 64, 64, None),
        "tq_decode_attention_latent": lambda: native.tq_decode_attention_latent(None, 0, 0, 0, 0, 1, 1, 512, 16, 1, 1, 1.0, 0, 0, 0,
                                                                                None),
        "tq_prefill_attention_latent": lambda: native.tq_prefill_attention_latent(None, 0, 0, 0, 0, 1, 1, 1, 512, 16, 1, 1, 1.0, 0, 0,
                                                                                  0, None),
    }
    for name, call in calls.items():
        with pytest.raises(native.TQError) as e:
            call()
        assert e.value.status == native.TQ_ERR_INVALID_ARG and name in str(e.value) and "NULL" in str(e.value)
    assert native.tq_workspace_bytes_latent(None, 1, 1, 1, 512) == 0


def _codec(device):
    c = Codec.__new__(Codec)
    c.head_dim, c.device, c.handle = 128, device, None
    return c


def test_wrapper_refuses_before_any_call(monkeypatch):
    """Shapes, types and devices are checked before the library is called (no handle is needed to refuse)."""
    monkeypatch.setattr(Codec, "_elsewhere", lambda self, stream: False)
    c = _codec(-1)  # get_device() of a CPU tensor: everything but the device is right in the calls below
    lat, key = torch.zeros(3, 256, dtype=torch.bfloat16), torch.zeros(3, 64, dtype=torch.bfloat16)
    s, pool = torch.zeros(3, dtype=torch.int64), torch.zeros(2, 16, 320, dtype=torch.bfloat16)
    q, rope = torch.zeros(3, 5, 64, dtype=torch.bfloat16), torch.zeros(4, 64)
    for bad in (dict(latent=lat.float()), dict(latent=lat[0]), dict(k_rope=key[:2]), dict(k_rope=key[:, :32]), dict(slot_mapping=s.int()),
                dict(pool=pool.float()), dict(pool=pool[:1]), dict(pool=pool[..., :256]), dict(q=q[0]), dict(q=q[:2]), dict(q_out=q),
                dict(q=q, q_out=q.float()), dict(q=q, q_out=q[:, :4]), dict(q=q[..., :32]), dict(q=q.repeat(1, 1, 2)[..., ::2]),
                dict(latent=lat.T.contiguous().T), dict(rope=rope), dict(rope=rope, positions=s.int()), dict(rope=rope[:, :32], positions=s),
                dict(rope=rope.double(), positions=s), dict(rope=rope[0], positions=s), dict(norm_weight=torch.ones(256)),
                dict(norm_weight=torch.ones(64, dtype=torch.bfloat16)), dict(num_blocks=3)):
        a = dict(latent=lat, k_rope=key, slot_mapping=s, pool=pool, page_size=16, num_blocks=2)
        a.update(bad)
        with pytest.raises(ValueError):
            c.append_latent(**a)
    query, lens, table = torch.zeros(1, 4, 320, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32)
    ws = torch.zeros(16, dtype=torch.uint8)
    for bad in (dict(q=query.float()), dict(q=query[..., :256]), dict(q=query[0]), dict(block_table=table.long()), dict(block_table=table[0]),
                dict(seq_lens=lens.long()), dict(seq_lens=torch.zeros(2, dtype=torch.int32)), dict(pool=pool[:1]), dict(workspace=ws[::2]),
                dict(out=query), dict(out=query[..., :256].float())):
        a = dict(q=query, pool=pool, block_table=table, seq_lens=lens, page_size=16, num_blocks=2, sm_scale=0.1, workspace=ws)
        a.update(bad)
        with pytest.raises(ValueError):
            c.decode_attention_latent(**a)
    with pytest.raises(ValueError):
        c.prefill_attention_latent(query, pool, table, lens, 16, 2, 0.1)
    c.device = 0  # tensors that are not on the handle's device
    with pytest.raises(ValueError, match="cuda:0"):
        c.append_latent(lat, key, s, pool, 16, 2)
    with pytest.raises(ValueError, match="cuda:0"):
        c.decode_attention_latent(query, pool, table, lens, 16, 2, 0.1)


def test_a_stream_of_another_device_is_refused():
    c = _codec(0)
    other = types.SimpleNamespace(cuda_stream=5, device=torch.device("cuda", 1))
    x, s = torch.zeros(1, 320, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int64)
    pool, i32 = torch.zeros(1, 16, 320, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: c.append_latent(x[:, :256], x[:, 256:], s, pool, 16, 1, stream=other),
                 lambda: c.decode_attention_latent(x[:, None], pool, i32[None], i32, 16, 1, 0.1, stream=other),
                 lambda: c.prefill_attention_latent(x[:, None, None], pool, i32[None], i32, 16, 1, 0.1, stream=other)):
        with pytest.raises(ValueError, match="stream"):
            call()


def test_reference_attention():
    g = torch.Generator().manual_seed(0)
    pool, table = torch.randn(3, 16, 128, generator=g).double(), torch.tensor([[2, 0]])
    q = torch.randn(1, 2, 3, 128, generator=g).double()
    out, bound = R.attention(q, pool, table, [20], 16, 0.2)
    k = torch.cat([pool[2], pool[0]])[:20]
    for i, n in ((0, 19), (1, 20)):
        want = torch.softmax(q[0, i] @ k[:n].T * 0.2, -1) @ k[:n, :64]
        assert torch.allclose(out[0, i], want, rtol=1e-12, atol=1e-12)
    assert bool((bound > 0).all())


def test_reference_norm_and_rotation():
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn(4, 256, generator=g), torch.randn(256, generator=g)
    y = R.norm(x, w, 0.0)
    assert torch.allclose((y / w.double()).norm(dim=1), torch.full((4,), 16.0, dtype=torch.float64))
    v = torch.randn(3, 2, 64, generator=g)
    ang = torch.rand(5, 32, generator=g)
    rope = torch.cat([ang.cos(), ang.sin()], 1)
    for inter in (False, True):
        r = R.rotate(v, rope, torch.tensor([0, 4, 2]), inter)
        assert torch.allclose(r.norm(dim=-1), v.norm(dim=-1), rtol=1e-6)
        back = R.rotate(r, torch.cat([ang.cos(), -ang.sin()], 1), torch.tensor([0, 4, 2]), inter)
        assert torch.allclose(back, v, atol=1e-6)
