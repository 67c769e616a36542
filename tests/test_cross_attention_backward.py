"""Gradients of the attention to an encoder's states: refusals (host checks, no CUDA call) and, on a
GPU, parity with the formulas in 64 bits and with differences."""
import ctypes
import math

import pytest
import torch

import sparse_mixed_precision_b200 as da2
from tests.test_cross_attention import DT, check_out, formulas64, heads, make


# ------------------------------------------------------------------ refusals, no GPU
def _status(cfg, dk=(0x1000, None), lse=0x1000, ws=0x1000, ws_bytes=1 << 40):
    from sparse_mixed_precision_b200.block_ops import Tensor

    def t(H, T, spec=(0x1000, None)):
        return ctypes.byref(Tensor(spec[0], *(spec[1] or (H * T * cfg.d, T * cfg.d, cfg.d))))

    q, k = (cfg.H, cfg.Tq), (max(cfg.Hkv, 1), cfg.Tk)
    return da2.lib().da2_cross_attention_backward(ctypes.byref(cfg), t(*q), t(*q), t(*k), t(*k), t(*q), lse, None,
                                                  t(*q), t(*k, dk), t(*k), ws, ws_bytes, None)


def test_bad_arguments_are_refused():
    c = da2.cross_config(2, 4, 300, 77, 64)
    need = da2.cross_attention_workspace_size(c, backward=True)
    assert need > 256 + 2 * 4 * 2 * 4 * 384
    assert _status(c, lse=None) == 1
    assert _status(c, lse=0x1002) == 3
    assert _status(c, dk=(None, None)) == 1
    assert _status(c, dk=(0x1000, (77 * 64 * 4, 0, 64))) == 1
    assert _status(c, dk=(0x1000, (77 * 64 * 4, 77 * 64, 68))) == 3
    assert _status(c, ws=None) == 1
    assert _status(c, ws=0x1080) == 3
    assert _status(c, ws_bytes=need - 1) == 4
    assert _status(da2.cross_config(2, 4, 300, 77, 96)) == 2
    assert _status(da2.cross_config(2, 4, 300, 77, 64, Hkv=3)) == 1
    x = torch.zeros(2, 4, 300, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="lse is needed"):
        da2.cross_attention_backward(c, x, x, x, x, x, None, x, x, x, x)


# ------------------------------------------------------------------ GPU
def gradients64(q, k, v, dout, lens, layout, dt, scale=None):
    """Gradients of the definition and, per element, how far the rounded operands may take them:
    p rounded once (half a step), dS once, out (an input of D) once; S, dP and D are fp32 sums."""
    q, k, v, do = (heads(x, layout).double() for x in (q, k, v, dout))
    B, H, Tq, d = q.shape
    Hkv, Tk = k.shape[1:3]
    rep = H // Hkv
    scale = 1 / math.sqrt(d) if scale is None else scale
    half = torch.finfo(dt).eps / 2
    tiny = 2.0 ** -31 if dt == torch.float16 else 0.0       # of p or dS below fp16's normals, scaled by 2^6
    g = [torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)]
    tol = [torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)]
    for b in range(B):
        n = Tk if lens is None else min(max(lens[b], 0), Tk)
        if n == 0:
            continue
        kb, vb = (x[b, :, :n].repeat_interleave(rep, 0) for x in (k, v))
        T = lambda x: x.transpose(1, 2)  # noqa: E731
        fold = lambda x: x.view(Hkv, rep, n, d).sum(1)  # noqa: E731
        s = q[b] @ T(kb) * scale
        s_err = (q[b].abs() @ T(kb.abs()) * scale).max() * 2.0 ** -21 + 2.0 ** -19
        p = torch.softmax(s, -1)
        o, dp = p @ vb, do[b] @ T(vb)
        delta = (do[b] * o).sum(-1, keepdim=True)
        ds = p * (dp - delta)
        absdp = do[b].abs() @ T(vb.abs())
        e_ds = ds.abs() * (half + 2 * s_err) + tiny + \
            p * ((do[b].abs() * o.abs()).sum(-1, keepdim=True) * (half + 2.0 ** -20) + absdp * 2.0 ** -20)
        e_p = p * (half * 1.01 + 2 * s_err) + tiny
        g[0][b], tol[0][b] = ds @ kb * scale, e_ds @ kb.abs() * scale
        g[1][b, :, :n], tol[1][b, :, :n] = fold(T(ds) @ q[b]) * scale, fold(T(e_ds) @ q[b].abs()) * scale
        g[2][b, :, :n], tol[2][b, :, :n] = fold(T(p) @ do[b]), fold(T(e_p) @ do[b].abs())
    return [(x, t + x.abs() * half + torch.finfo(dt).smallest_normal * half) for x, t in zip(g, tol)]


def check_grads(got, want, layout):
    for name, x, (ref, tol) in zip(("dq", "dk", "dv"), got, want):
        x = heads(x, layout).double()
        assert torch.isfinite(x).all(), name
        off = ((x - ref).abs() - tol).max().item()
        assert off <= 0, (name, off)


def run_both(cfg, q, k, v, dout, kv_len):
    out, lse = torch.empty_like(q), torch.empty(cfg.B, cfg.H, cfg.Tq, device="cuda")
    da2.cross_attention(cfg, q, k, v, out, da2.cross_attention_workspace(cfg, "cuda"), kv_len=kv_len, lse=lse)
    grads = [torch.full_like(x, 7.0) for x in (q, k, v)]
    ws = da2.cross_attention_workspace(cfg, "cuda", backward=True)
    da2.cross_attention_backward(cfg, dout, q, k, v, out, lse, *grads, ws, kv_len=kv_len)
    assert da2.cross_attention_get_error(ws) == 0
    again = [torch.empty_like(x) for x in (q, k, v)]
    da2.cross_attention_backward(cfg, dout, q, k, v, out, lse, *again, ws, kv_len=kv_len)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))      # fixed order of the sums
    return out, lse, grads


CASES = [  # B, H, Hkv, Tq, Tk, d, lens
    (1, 1, 1, 1, 1, 64, None), (1, 2, 2, 128, 128, 128, None), (1, 1, 1, 129, 16, 128, None),
    (2, 3, 3, 257, 77, 64, [77, 5]), (1, 2, 1, 300, 257, 128, [257]), (2, 4, 2, 511, 512, 128, [512, 129]),
    (3, 2, 2, 640, 300, 128, [0, 300, 17]), (2, 2, 2, 64, 129, 64, [128, 1]), (1, 20, 20, 1000, 512, 128, None),
    (2, 24, 24, 700, 256, 128, [182, 35]), (1, 5, 1, 1, 2100, 128, None), (2, 40, 8, 3, 1000, 128, [1000, 131]),
    (4, 3, 3, 7, 2049, 64, [0, 2049, 1, 1500]), (1, 1, 1, 9000, 130, 64, [129]), (1, 150, 150, 40, 250, 128, None),
    (2, 2, 2, 100, 100, 128, [0, 0]), (3, 60, 60, 260, 130, 64, [130, 0, 129]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("layout", ["bhtd", "bthd"])
def test_gradients_match_the_formulas(case, dtype, layout):
    B, H, Hkv, Tq, Tk, d, lens = case
    dt = DT[dtype]
    q, k, v, kv_len = make(B, H, Hkv, Tq, Tk, d, dt, layout, lens, wide=Tq % 2 == 1)
    g = torch.Generator(device="cuda").manual_seed(9)
    dout = torch.randn(q.shape, generator=g, device="cuda").to(dt)
    cfg = da2.cross_config(B, H, Tq, Tk, d, Hkv=Hkv, dtype=dt, layout=layout)
    out, lse, grads = run_both(cfg, q, k, v, dout, kv_len)
    check_out(out, lse, formulas64(q, k, v, lens, layout), dt, layout)
    check_grads(grads, gradients64(q, k, v, dout, lens, layout, dt), layout)


@pytest.mark.gpu
def test_gradients_match_differences():
    """Central differences of the 64-bit forward formula along random directions, against the fp16
    gradients: the tolerance is the one of the formulas, summed over the direction."""
    B, H, Hkv, Tq, Tk, d = 1, 2, 1, 37, 70, 64
    q, k, v, kv_len = make(B, H, Hkv, Tq, Tk, d, torch.float16, "bhtd", [61], behind="inf")
    k[:, :, 61:], v[:, :, 61:] = 0, 0
    dout = torch.randn(q.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)).half()
    cfg = da2.cross_config(B, H, Tq, Tk, d, Hkv=Hkv, dtype=torch.float16)
    _, _, grads = run_both(cfg, q, k, v, dout, kv_len)
    want = gradients64(q, k, v, dout, [61], "bhtd", torch.float16)
    f = lambda *x: (formulas64(*x, [61], "bhtd")[0] * dout.double()).sum()  # noqa: E731
    base = [x.double() for x in (q, k, v)]
    gen = torch.Generator(device="cuda").manual_seed(8)
    for i in range(3):
        for _ in range(3):
            u = torch.randn(base[i].shape, generator=gen, device="cuda", dtype=torch.float64)
            h = 1e-4
            up, dn = list(base), list(base)
            up[i], dn[i] = base[i] + h * u, base[i] - h * u
            num = (f(*up) - f(*dn)) / (2 * h)
            off = (want[i][1] * u.abs()).sum() + 1e-6 * (want[i][0].abs() * u.abs()).sum()
            assert (num - (grads[i].double() * u).sum()).abs() <= off


@pytest.mark.gpu
def test_slices_scale_and_graph():
    """Fused key/value slices and their fused gradient; a scale of its own; a captured pass of both
    directions replayed with other inputs and lengths."""
    B, H, Tq, Tk, d = 2, 3, 260, 200, 128
    gen = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    kv, q, dout = rnd(B, Tk, 2, H, d), rnd(B, Tq, H, d), rnd(B, Tq, H, d)
    dkv, dq, out = torch.empty_like(kv), torch.empty_like(q), torch.empty_like(q)
    lse = torch.empty(B, H, Tq, device="cuda")
    lens = torch.tensor([200, 131], dtype=torch.int32, device="cuda")
    cfg = da2.cross_config(B, H, Tq, Tk, d, layout="bthd", sm_scale=0.2)
    ws, wsb = da2.cross_attention_workspace(cfg, "cuda"), da2.cross_attention_workspace(cfg, "cuda", backward=True)

    def both():
        da2.cross_attention(cfg, q, kv[:, :, 0], kv[:, :, 1], out, ws, kv_len=lens, lse=lse)
        da2.cross_attention_backward(cfg, dout, q, kv[:, :, 0], kv[:, :, 1], out, lse, dq, dkv[:, :, 0], dkv[:, :, 1],
                                     wsb, kv_len=lens)

    def check(n):
        check_grads((dq, dkv[:, :, 0], dkv[:, :, 1]),
                    gradients64(q, kv[:, :, 0], kv[:, :, 1], dout, n, "bthd", torch.bfloat16, 0.2), "bthd")

    both()
    check([200, 131])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    q.copy_(rnd(B, Tq, H, d))
    lens.copy_(torch.tensor([77, 0], dtype=torch.int32))
    graph.replay()
    check([77, 0])


@pytest.mark.gpu
def test_wait_that_runs_out_is_reported():
    q, k, v, _ = make(1, 2, 2, 300, 200, 128, torch.bfloat16, "bhtd", None)
    cfg = da2.cross_config(1, 2, 300, 200, 128)
    dout = torch.randn_like(q)
    out, lse, grads = run_both(cfg, q, k, v, dout, None)
    stalled = da2.cross_config(1, 2, 300, 200, 128, flags=da2.FLAG_TEST_STALL)
    ws = da2.cross_attention_workspace(stalled, "cuda", backward=True)
    bad = [torch.empty_like(x) for x in grads]
    da2.cross_attention_backward(stalled, dout, q, k, v, out, lse, *bad, ws)
    assert da2.cross_attention_get_error(ws) == 1
    da2.cross_attention_backward(cfg, dout, q, k, v, out, lse, *bad, ws)
    assert da2.cross_attention_get_error(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(grads, bad))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: the last rows of the last head, both directions."""
    B, H, Tq, Tk, d = 4, 40, 118800, 40, 128
    gen = torch.Generator(device="cuda").manual_seed(6)
    q = torch.empty(B, H, Tq, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    k, v = (torch.empty(B, H, Tk, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(2))
    cfg = da2.cross_config(B, H, Tq, Tk, d)
    out, lse = torch.empty_like(q), torch.empty(B, H, Tq, device="cuda")
    da2.cross_attention(cfg, q, k, v, out, da2.cross_attention_workspace(cfg, "cuda"), lse=lse)
    last = (slice(B - 1, B), slice(H - 1, H))
    cut = (*last, slice(Tq - 300, Tq))
    want = formulas64(q[cut], k[last], v[last], None, "bhtd")
    check_out(out[cut], lse[cut[:2]][:, :, -300:], want, torch.bfloat16, "bhtd")
    # the gradient of out is zero but in the rows that are compared: dk and dv come from them alone
    dout = torch.zeros_like(q)
    dout[cut] = torch.randn(1, 1, 300, d, generator=gen, device="cuda").to(torch.bfloat16)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = da2.cross_attention_workspace(cfg, "cuda", backward=True)
    da2.cross_attention_backward(cfg, dout, q, k, v, out, lse, dq, dk, dv, ws)
    grads = gradients64(q[cut], k[last], v[last], dout[cut], None, "bhtd", torch.bfloat16)
    check_grads((dq[cut], dk[last], dv[last]), grads, "bhtd")
    assert (dq[0, 0] == 0).all() and (dk[0] == 0).all() and (dv[0] == 0).all()
