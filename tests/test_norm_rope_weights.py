"""Where the weights of the norm and their gradients may lie in a flat fp32 buffer."""
import ctypes

import pytest
import torch

import sparse_mixed_precision_b200 as da2
from tests.test_norm_rope import _make


def test_alignment_of_weights_and_their_gradients():
    """Weights are read 16 bytes at a time, their gradients written a float at a time."""
    from sparse_mixed_precision_b200.block_ops import Tensor
    cfg = da2.norm_rope_config(1, 2, 2, 5, 64, T_rot=0)
    t, L = ctypes.byref(Tensor(0x1000, 640, 320, 64)), da2.lib()
    for w in (0x1002, 0x1004, 0x1008):
        assert L.da2_qk_norm_rope(ctypes.byref(cfg), t, t, w, None, None, None, t, t, None) == 3
        assert L.da2_qk_norm_rope(ctypes.byref(cfg), t, t, None, w, None, None, t, t, None) == 3
    back = lambda dwq, dwk, n, w=None: L.da2_qk_norm_rope_backward(  # noqa: E731
        ctypes.byref(cfg), t, t, t, t, w, None, None, None, t, t, dwq, dwk, 0x1000, n, None)
    assert back(0x1002, None, 1 << 30) == 3 and back(None, 0x1006, 1 << 30) == 3
    assert back(0x1004, 0x100c, 1 << 30, w=0x1004) == 3
    assert back(0x1004, 0x100c, 16) == 4                # aligned well enough: only the workspace is too small


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("offset", [1, 2, 7])
def test_weight_gradients_at_odd_offsets(d, offset):
    """Into a flat gradient buffer: the same bits as elsewhere, nothing beside them."""
    B, H, T = 2, 3, 50
    q, k, wq, wk, cos, sin = _make(B, H, H, T, d, torch.bfloat16, "bthd", T)
    cfg = da2.norm_rope_config(B, H, H, T, d, layout="bthd")
    flat = torch.full((2 * d + offset + 9,), 9.0, device="cuda")
    ws = da2.qk_norm_rope_workspace(cfg, "cuda")
    res = []
    for dwq, dwk in (torch.empty(2, d, device="cuda"), flat[offset:offset + 2 * d].view(2, d)):
        dx = [torch.empty_like(q) for _ in range(2)]
        da2.qk_norm_rope_backward(cfg, q, k, q, k, wq, wk, cos, sin, *dx, dwq, dwk, ws)
        res.append([*dx, dwq.clone(), dwk.clone()])
    assert all(torch.equal(a, b) for a, b in zip(*res))
    assert (flat[:offset] == 9.0).all() and (flat[offset + 2 * d:] == 9.0).all()
