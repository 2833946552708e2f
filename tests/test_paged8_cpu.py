"""The references for 8-bit pages against torch's own e4m3 type, and refusals that need no GPU."""
import numpy as np
import pytest
import torch

import paged8 as R
from rotated_codebook_kv_gb300 import Codec, build, native


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return native.load()


def test_e4m3_values_and_rounding():
    codes = torch.arange(256).to(torch.uint8)
    assert np.array_equal(codes.view(torch.float8_e4m3fn).double().numpy(), R.E4M3, equal_nan=True)
    g = torch.Generator().manual_seed(0)
    x = torch.cat([torch.randn(20000, generator=g) * 2.0 ** torch.randint(-12, 8, (20000,), generator=g),
                   torch.tensor(R.E4M3[:127]), -torch.tensor(R.E4M3[:127]),
                   torch.tensor((R.E4M3[:126] + R.E4M3[1:127]) / 2)]).float().clamp(-448, 448)
    assert np.array_equal(R.e4m3_codes(x.double().numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert R.e4m3_codes(np.array([1e9, -1e9, np.inf, np.nan])).tolist() == [0x7E, 0xFE, 0x7E, 0x7F]


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.5, 1), (224.0, -1), (1.75, -8), (1.7500001, -7), (0.0, -100),
                                    (1e-40, -100), (3.38e38, 120)])
def test_page_scale(amax, e):
    assert R.page_scale(amax) == 2.0 ** e


def test_null_handle_refused():
    calls = {
        "tq_append_kv_bf16": lambda: native.tq_append_kv_bf16(None, 0, 0, 0, 1, 0, 1, 0, 128, 128, 0, 0, 0, 0, 0, 0, 0,
                                                              0, 16, 1, 0, None),
        "tq_append_kv_fp8": lambda: native.tq_append_kv_fp8(None, 0, 0, 0, 1, 0, 1, 0, 128, 128, 0, 0, 0, 0, 0, 0, 0, 0,
                                                            0, 0, 16, 1, 0, None),
        "tq_decode_attention_fp8": lambda: native.tq_decode_attention_fp8(None, 0, 0, 0, 0, 0, 0, 0, 1, 1, 1, 16, 1, 1,
                                                                          1.0, 1, 0, 0, 0, None),
        "tq_prefill_attention_fp8": lambda: native.tq_prefill_attention_fp8(None, 0, 0, 0, 0, 0, 0, 0, 1, 1, 1, 1, 16, 1,
                                                                            1, 1.0, 1, 0, 0, 0, None),
    }
    for name, call in calls.items():
        with pytest.raises(native.TQError) as e:
            call()
        assert e.value.status == native.TQ_ERR_INVALID_ARG and name in str(e.value) and "NULL" in str(e.value)
    assert native.tq_decode_splits_fp8(None, 1, 1, 1, 16) == 1
    assert native.tq_prefill_splits_fp8(None, 1, 1, 1, 1, 1, 16) == 1
    assert native.tq_workspace_bytes_fp8(None, 1, 1, 2) == 0


def test_wrapper_refuses_before_any_call(monkeypatch):
    """Shapes, types and devices are checked before the library is called (no handle is needed to refuse)."""
    monkeypatch.setattr(Codec, "_elsewhere", lambda self, stream: False)
    c = Codec.__new__(Codec)
    c.head_dim, c.device, c.handle = 128, 0, None
    x = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    s = torch.zeros(3, dtype=torch.int64)
    rope = torch.zeros(4, 64)
    pool = torch.zeros(2, 2, 16, 128, dtype=torch.uint8).view(torch.float8_e4m3fn)
    sc = torch.ones(2, 2)
    c.device = -1  # get_device() of a CPU tensor: everything but the device is right in the calls below
    assert c._flat(sc, torch.float32, 4, "x") == sc.data_ptr() and c._rows(x, 3, 2, "x") == (x.data_ptr(), 256)
    for bad in (dict(v=x[:2]), dict(k=x.float(), v=x.float()), dict(s=s.int()), dict(s=s[:2]), dict(q=x[:2]),
                dict(q_out=x), dict(q=x, q_out=x.float()), dict(rope=rope), dict(rope=rope, positions=s.int()),
                dict(rope=rope.double(), positions=s), dict(rope=rope[0], positions=s),
                dict(k=x.transpose(0, 1), v=x.transpose(0, 1)), dict(k=x[0], v=x[0]), dict(kp=pool.view(torch.uint8)),
                dict(nb=3), dict(ks=sc.double()), dict(ks=sc[:1]), dict(k=x.repeat(1, 1, 2)[:, :, ::2])):
        a = dict(k=x, v=x, s=s, kp=pool, ks=sc, nb=2)
        a.update({k: v for k, v in bad.items() if k in a})
        more = {k: v for k, v in bad.items() if k not in a}
        with pytest.raises(ValueError):
            c.append_kv_fp8(a["k"], a["v"], a["s"], a["kp"], pool, a["ks"], sc, 16, a["nb"], **more)
    q, lens, table = torch.zeros(1, 4, 128, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32)
    for bad in (dict(q=q.float()), dict(q=q[..., :64]), dict(block_table=table.long()), dict(seq_lens=lens.long()),
                dict(seq_lens=torch.zeros(2, dtype=torch.int32)), dict(q=q[0]), dict(block_table=table[0])):
        a = dict(q=q, block_table=table, seq_lens=lens)
        a.update(bad)
        with pytest.raises(ValueError):
            c.decode_attention_fp8(a["q"], pool, pool, sc, sc, a["block_table"], a["seq_lens"], 2, 16, 2, 0.1)
    with pytest.raises(ValueError):
        c.prefill_attention_fp8(q, pool, pool, sc, sc, table, lens, 2, 16, 2, 0.1)
    c.device = 0  # tensors that are not on the handle's device
    with pytest.raises(ValueError, match="cuda:0"):
        c.append_kv_fp8(x, x, s, pool, pool, sc, sc, 16, 2)
    with pytest.raises(ValueError, match="cuda:0"):
        c.decode_attention_fp8(q, pool, pool, sc, sc, table, lens, 2, 16, 2, 0.1)
