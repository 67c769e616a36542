"""The operators of one video-DiT block together, as a model runs them: norm and rotation of the
queries and keys, the sparse self-attention, the norm of the second queries and keys, the attention
to the encoder's states, and the gradients of that branch."""
import pytest
import torch

import sparse_mixed_precision_b200 as da2
from sparse_mixed_precision_b200.synth import WORKLOADS, generate
from tests.test_cross_attention import check_out, formulas64
from tests.test_cross_attention_backward import check_grads, gradients64
from tests.test_norm_rope import _close, _forward64


def rope_tables(w):
    """cos and sin [T, d/2] of the video's frame, row and column axes."""
    t = torch.arange(w.T, device="cuda")
    axes = (t // (w.Hf * w.Wf), t // w.Wf % w.Hf, t % w.Wf)
    n = w.d // 2
    parts = (n - 2 * (n // 3), n // 3, n // 3)
    ang = torch.cat([a.double()[:, None] * 10000.0 ** (-torch.arange(p, device="cuda").double() / p)
                     for a, p in zip(axes, parts)], 1)
    return ang.cos().float(), ang.sin().float()


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["bhtd", "bthd"])
@pytest.mark.parametrize("captured", [False, True])
def test_block(layout, captured):
    w = WORKLOADS["tiny"]
    B, H, T, d, L = w.B, w.H, w.T, w.d, 77
    flags = da2.FLAG_LAYOUT_BTHD if layout == "bthd" else 0
    heads = lambda x: x.transpose(1, 2) if layout == "bthd" else x  # noqa: E731
    q, k, v = (heads(x).contiguous() for x in generate(w, device="cuda"))
    gen = torch.Generator(device="cuda").manual_seed(1)
    shape = (B, L, H, d) if layout == "bthd" else (B, H, L, d)
    kc, vc = (torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    wq, wk = (1 + 0.1 * torch.randn(d, generator=gen, device="cuda") for _ in range(2))
    cos, sin = rope_tables(w)
    lens = torch.tensor([61], dtype=torch.int32, device="cuda")
    dout = torch.randn(q.shape, generator=gen, device="cuda").to(torch.bfloat16)

    cfg = da2.config(w, flags=flags)
    ncfg = da2.norm_rope_config(B, H, H, T, d, layout=layout)
    qcfg = da2.norm_rope_config(B, H, 0, T, d, T_rot=0, layout=layout)
    kcfg = da2.norm_rope_config(B, H, 0, L, d, T_rot=0, layout=layout)
    xcfg = da2.cross_config(B, H, T, L, d, layout=layout)
    ws = torch.empty(da2.workspace_size(cfg), dtype=torch.uint8, device="cuda")
    xws = da2.cross_attention_workspace(xcfg, "cuda")
    xwb = da2.cross_attention_workspace(xcfg, "cuda", backward=True)
    nws = da2.qk_norm_rope_workspace(qcfg, "cuda")
    qn, kn, sa, q2, k2, ca, dq2, dk2, dv2, dsa = (torch.empty_like(x) for x in (q, k, q, q, kc, q, q, kc, vc, q))
    lse, dw = torch.empty(B, H, T, device="cuda"), torch.empty(d, device="cuda")

    def block():
        da2.qk_norm_rope(ncfg, q, k, wq, wk, cos, sin, qn, kn)
        da2.forward(cfg, qn, kn, v, sa, ws)
        da2.qk_norm_rope(qcfg, sa, None, wq, None, None, None, q2, None)
        da2.qk_norm_rope(kcfg, kc, None, wk, None, None, None, k2, None)
        da2.cross_attention(xcfg, q2, k2, vc, ca, xws, kv_len=lens, lse=lse)
        da2.cross_attention_backward(xcfg, dout, q2, k2, vc, ca, lse, dq2, dk2, dv2, xwb, kv_len=lens)
        da2.qk_norm_rope_backward(qcfg, dq2, None, sa, None, wq, None, None, None, dsa, None, dw, None, nws)

    if captured:
        block()                                         # loads the kernels before the capture
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            block()
        for x in (qn, kn, sa, q2, k2, ca, dq2, dk2, dv2, dsa):
            x.zero_()
        graph.replay()
    else:
        block()
    torch.cuda.synchronize()
    assert da2.get_error(cfg, ws) == 0
    assert da2.cross_attention_get_error(xws) == 0 and da2.cross_attention_get_error(xwb) == 0

    bf = torch.bfloat16
    c3, s3 = cos[None], sin[None]
    none = torch.ones(1, 0, d // 2, device="cuda")
    _close(heads(qn), _forward64(heads(q), wq, c3, s3, False, 1e-6), bf)
    _close(heads(kn), _forward64(heads(k), wk, c3, s3, False, 1e-6), bf)
    # the self-attention takes the rotated tensors as it takes any others: the other layout's call on
    # the same values gives the same bits
    other = da2.config(w, flags=da2.FLAG_LAYOUT_BTHD ^ flags)
    swap = lambda x: x.transpose(1, 2).contiguous()  # noqa: E731
    ref = torch.empty_like(swap(sa))
    da2.forward(other, swap(qn), swap(kn), swap(v), ref, ws)
    assert torch.equal(swap(ref), sa)
    _close(heads(q2), _forward64(heads(sa), wq, none, none, False, 1e-6), bf)
    check_out(ca, lse, formulas64(q2, k2, vc, [61], layout), bf, layout)
    check_grads((dq2, dk2, dv2), gradients64(q2, k2, vc, dout, [61], layout, bf), layout)
    x64 = heads(sa).double().requires_grad_()
    w64 = wq.double().requires_grad_()
    gx, gw = torch.autograd.grad(_forward64(x64, w64, none, none, False, 1e-6), (x64, w64), heads(dq2).double())
    _close(heads(dsa), gx, bf, extra=2.0 ** -18)
    # fp32 sums of T H terms in chains of fewer than 300, each rounding 2^-24 of the absolute sum
    n64 = x64.detach() / torch.sqrt((x64.detach() ** 2).mean(-1, keepdim=True) + 1e-6)
    assert ((dw.double() - gw).abs() <= (heads(dq2).double() * n64).abs().sum((0, 1, 2)) * 2.0 ** -24 * 300).all()
