"""Latent pages at the ends of their ranges, on both of the attention's kernels."""
import pytest
import torch

from rotated_codebook_kv_gb300 import Codec, native
from test_gpu_latent import DEV, case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dl,Tq", [(512, 64), (256, 64), (512, 128), (256, 128)])
def test_the_join_waits_no_longer_than_the_wait_limit(dl, Tq):
    """A long sequence cut into many pieces; a NaN in its last token keeps the worker of the last piece for some 50 to 200 us
    (it looks for the rows that see it), while the others wait for it to join them: longer than a limit of 20 us, which the
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
    own.set_wait_limit(40000)
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
