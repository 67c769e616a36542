"""Attention to an encoder's states at the places where it once went wrong: short keys over many query
tiles, gradients over fp16's range, long batches, parts without weight, aborted calls."""
import pytest
import torch

import sparse_mixed_precision_b200 as da2
from tests.test_cross_attention import make
from tests.test_cross_attention_backward import check_grads, gradients64, run_both


@pytest.mark.gpu
@pytest.mark.parametrize("Tk,lens", [(77, None), (128, [128, 1, 0, 65]), (300, [128, 300, 17, 129])])
def test_many_query_tiles_of_one_key_tile(Tk, lens):
    """Blocks that walk many query tiles whose keys fit one tile, alone and between items of several:
    each item's loads wait for all of the item before. Equal bits over repeated calls, and parity."""
    B, H, Tq, d = 4 if lens else 1, 24, 4000, 64
    q, k, v, kv_len = make(B, H, H, Tq, Tk, d, torch.bfloat16, "bhtd", lens, seed=3)
    dout = torch.randn(q.shape, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(q.dtype)
    cfg = da2.cross_config(B, H, Tq, Tk, d)
    out, lse, grads = run_both(cfg, q, k, v, dout, kv_len)
    check_grads(grads, gradients64(q, k, v, dout, lens, "bhtd", torch.bfloat16), "bhtd")
    ws = da2.cross_attention_workspace(cfg, "cuda", backward=True)
    for _ in range(20):
        again = [torch.empty_like(x) for x in grads]
        da2.cross_attention_backward(cfg, dout, q, k, v, out, lse, *again, ws, kv_len=kv_len)
        assert all(torch.equal(a, b) for a, b in zip(grads, again))
    assert da2.cross_attention_get_error(ws) == 0
