"""Streams given to the calls over plain and 8-bit pages: refusals that need no GPU."""
import types

import pytest
import torch

from rotated_codebook_kv_gb300 import Codec


def test_a_stream_of_another_device_is_refused():
    """It was passed over: the work went to the current stream of the Codec's device, unordered with the one given."""
    c = Codec.__new__(Codec)
    c.head_dim, c.device, c.handle = 128, 0, None
    other = types.SimpleNamespace(cuda_stream=5, device=torch.device("cuda", 1))
    x = torch.zeros(1, 2, 128, dtype=torch.bfloat16)
    s = torch.zeros(1, dtype=torch.int64)
    pool, sc = torch.zeros(1, 2, 16, 128, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.ones(1, 2)
    i32 = torch.zeros(1, dtype=torch.int32)
    calls = [lambda: c.append_kv_bf16(x, x, s, pool, pool, 16, 1, stream=other),
             lambda: c.append_kv_fp8(x, x, s, pool, pool, sc, sc, 16, 1, stream=other),
             lambda: c.decode_attention_fp8(x, pool, pool, sc, sc, i32[None], i32, 2, 16, 1, 0.1, stream=other),
             lambda: c.prefill_attention_fp8(x[None], pool, pool, sc, sc, i32[None], i32, 2, 16, 1, 0.1, stream=other)]
    for call in calls:
        with pytest.raises(ValueError, match="stream"):
            call()
