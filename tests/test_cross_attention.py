"""Attention to an encoder's states, forward: refusals (host checks, no CUDA call) and, on a GPU,
parity with the formulas in 64 bits at the sizes, lengths and masks where it can go wrong."""
import ctypes
import math

import pytest
import torch

import sparse_mixed_precision_b200 as da2

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ refusals, no GPU
def _cfg(**kw):
    base = dict(B=2, H=4, Tq=300, Tk=77, d=64)
    base.update(kw)
    return da2.cross_config(**base)


def _status(cfg, q=(0x1000, None), k=(0x1000, None), out=(0x1000, None), ws=0x1000, ws_bytes=1 << 40, kv_len=None):
    """Status of a call whose pointers are never read: every refusal comes before the launch."""
    from sparse_mixed_precision_b200.block_ops import Tensor

    def t(spec, H, T):
        data, strides = spec
        return ctypes.byref(Tensor(data, *(strides or (H * T * cfg.d, T * cfg.d, cfg.d))))

    Hkv = max(cfg.Hkv, 1)
    return da2.lib().da2_cross_attention(ctypes.byref(cfg), t(q, cfg.H, cfg.Tq), t(k, Hkv, cfg.Tk),
                                         t((0x1000, None), Hkv, cfg.Tk), t(out, cfg.H, cfg.Tq), None, kv_len, ws,
                                         ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(H=0, Hkv=1), 1), (dict(Tq=0), 1), (dict(Tk=0), 1), (dict(Hkv=3), 1), (dict(Hkv=0), 1),
    (dict(sm_scale=-1.0), 1), (dict(sm_scale=float("inf")), 1), (dict(sm_scale=float("nan")), 1), (dict(flags=1), 1),
    (dict(d=96), 2), (dict(d=256), 2), (dict(B=1 << 16, H=1 << 12), 2), (dict(Tq=2147483647, H=64), 2),
])
def test_bad_configurations_are_refused(kw, status):
    c = _cfg(**kw)
    assert _status(c) == status
    n = ctypes.c_size_t()
    assert da2.lib().da2_cross_attention_workspace_size(ctypes.byref(c), ctypes.byref(n)) == status


def test_bad_arguments_are_refused():
    c = _cfg()
    assert _status(c, q=(None, None)) == 1
    assert _status(c, q=(0x1008, None)) == 3
    assert _status(c, k=(0x1000, (0, 77 * 64, 64))) == 1           # keys broadcast over the batch
    assert _status(c, out=(0x1000, (4 * 300 * 64, 300 * 64, 68))) == 3
    assert _status(c, out=(0x1000, (4 * 300 * 64, 300 * 64, 56))) == 1   # rows would overlap
    assert _status(c, ws=None) == 1
    assert _status(c, ws=0x1010) == 3
    assert _status(c, ws_bytes=0) == 4
    assert _status(c, kv_len=0x1002) == 3
    c.dtype = 2
    assert _status(c) == 1
    few = _cfg(Tq=1, Tk=4096)                                      # split over the keys: larger workspace
    assert da2.cross_attention_workspace_size(few) > 256
    assert _status(few, ws_bytes=256) == 4
    assert da2.cross_attention_workspace_size(_cfg()) == 256
    assert da2.lib().da2_cross_attention_get_error(None, 0, None, None) == 1


def test_binding_checks_tensors():
    cfg = _cfg()
    q, k = torch.zeros(2, 4, 300, 64, dtype=torch.bfloat16), torch.zeros(2, 4, 77, 64, dtype=torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        da2.cross_attention(cfg, q, k, k, q, ws)
    with pytest.raises(ValueError, match="q has shape"):
        da2.cross_attention(cfg, k, k, k, q, ws)
    with pytest.raises(ValueError, match="dtype"):
        da2.cross_attention(cfg, q.float(), k, k, q, ws)
    with pytest.raises(ValueError, match="CUDA tensor"):
        da2.cross_attention_get_error(ws)
    with pytest.raises(ValueError, match="dtype"):
        da2.cross_config(1, 1, 1, 1, 64, dtype=torch.float32)


# ------------------------------------------------------------------ GPU
def make(B, H, Hkv, Tq, Tk, d, dt, layout, lens, seed=0, wide=False, behind="nan", sharp=1.5):
    """q, k, v and the lengths; keys and values behind a length hold NaN or infinities."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def act(heads, T, scale=1.0):
        shape = (B, T, heads, d) if layout == "bthd" else (B, heads, T, d)
        if wide:
            x = torch.randn(shape[:2] + (shape[2] + 2, d + 24), generator=g, device="cuda") * scale
            return x.to(dt)[:, :, 1:-1, 8:-16]
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dt)

    q, k, v = act(H, Tq, sharp), act(Hkv, Tk), act(Hkv, Tk)
    kv_len = None
    if lens is not None:
        kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for b, n in enumerate(lens):
            for x, fill in ((k, math.nan if behind == "nan" else math.inf), (v, math.nan if behind == "nan" else -math.inf)):
                y = x[b].transpose(0, 1) if layout == "bthd" else x[b]
                y[:, max(n, 0):] = fill
    return q, k, v, kv_len


def heads(x, layout):
    return x.transpose(1, 2) if layout == "bthd" else x


def formulas64(q, k, v, lens, layout, scale=None):
    """out, lse, P and |v|-weighted sums of the definition, one batch entry at a time."""
    q, k, v = (heads(x, layout).double() for x in (q, k, v))
    B, H, Tq, d = q.shape
    rep, Tk = H // k.shape[1], k.shape[2]
    scale = 1 / math.sqrt(d) if scale is None else scale
    out, lse = torch.zeros_like(q), torch.full((B, H, Tq), -math.inf, dtype=torch.float64, device=q.device)
    pv = torch.zeros_like(q)
    smax = 0.0
    for b in range(B):
        n = Tk if lens is None else min(max(lens[b], 0), Tk)
        if n == 0:
            continue
        kb, vb = (x[b, :, :n].repeat_interleave(rep, 0) for x in (k, v))
        s = q[b] @ kb.transpose(1, 2) * scale
        lse[b] = torch.logsumexp(s, -1)
        p = torch.exp(s - lse[b][..., None])
        out[b], pv[b] = p @ vb, p @ vb.abs()
        smax = max(smax, (q[b].abs() @ kb.abs().transpose(1, 2) * scale).max().item())
    return out, lse, pv, smax


def check_out(out, lse, want, dt, layout):
    """P is rounded once, half a step relative to each p (fp16 below 2^-14: half of 2^-24, with
    the largest p of a row at least 1), the result once more; S is an fp32 sum of d products whose
    error, 2^-22 of the sum of their absolute values, shifts every exponent."""
    o64, lse64, pv, smax = want
    half = torch.finfo(dt).eps / 2
    s_err = smax * 2.0 ** -22 + 2.0 ** -20
    tol = o64.abs() * half + pv * (half * 1.01 + 2 * s_err) + 1e-6
    if dt == torch.float16:
        tol = tol + pv.amax() * 2.0 ** -25 * 5000
    got = heads(out, layout).double()
    assert torch.isfinite(got).all()
    off = ((got - o64).abs() - tol).max().item()
    assert off <= 0, off
    if lse is not None:
        assert torch.equal(torch.isinf(lse), torch.isinf(lse64))
        fin = torch.isfinite(lse64)
        assert ((lse.double() - lse64).abs()[fin] <= s_err + lse64.abs()[fin] * 2.0 ** -22 + 2.0 ** -20).all()


CASES = [  # B, H, Hkv, Tq, Tk, d, lens
    (1, 1, 1, 1, 1, 64, None), (1, 2, 2, 128, 128, 128, None), (1, 1, 1, 129, 16, 128, None),
    (2, 3, 3, 257, 77, 64, [77, 5]), (1, 2, 1, 300, 257, 128, [257]), (2, 4, 2, 511, 512, 128, [512, 129]),
    (3, 2, 2, 640, 300, 128, [0, 300, 17]), (2, 2, 2, 64, 129, 64, [128, 1]), (1, 40, 40, 1000, 512, 128, None),
    (2, 24, 24, 700, 256, 128, [182, 35]), (1, 5, 1, 1, 4096, 128, None), (2, 40, 8, 1, 1000, 128, [1000, 131]),
    (4, 3, 3, 7, 2049, 64, [0, 2049, 1, 1500]), (1, 8, 8, 33, 640, 128, [639]), (3, 60, 60, 520, 130, 64, [130, 0, 129]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("layout", ["bhtd", "bthd"])
def test_forward_matches_the_formula(case, dtype, layout):
    B, H, Hkv, Tq, Tk, d, lens = case
    dt = DT[dtype]
    q, k, v, kv_len = make(B, H, Hkv, Tq, Tk, d, dt, layout, lens, wide=Tq % 2 == 1)
    cfg = da2.cross_config(B, H, Tq, Tk, d, Hkv=Hkv, dtype=dt, layout=layout)
    ws = da2.cross_attention_workspace(cfg, "cuda")
    out = torch.full_like(q, 5.0)
    lse = torch.full((B, H, Tq), 5.0, device="cuda")
    da2.cross_attention(cfg, q, k, v, out, ws, kv_len=kv_len, lse=lse)
    assert da2.cross_attention_get_error(ws) == 0
    check_out(out, lse, formulas64(q, k, v, lens, layout), dt, layout)
    again = torch.empty_like(out)
    da2.cross_attention(cfg, q, k, v, again, ws, kv_len=kv_len)          # no lse, equal bits
    assert torch.equal(out, again)


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[130, 300], [0, 257]])
def test_infinities_behind_the_length_do_not_reach_the_result(lens):
    q, k, v, kv_len = make(2, 2, 2, 200, 300, 128, torch.bfloat16, "bhtd", lens, behind="inf")
    cfg = da2.cross_config(2, 2, 200, 300, 128)
    ws = da2.cross_attention_workspace(cfg, "cuda")
    out = torch.empty_like(q)
    da2.cross_attention(cfg, q, k, v, out, ws, kv_len=kv_len)
    check_out(out, None, formulas64(q, k, v, lens, "bhtd"), torch.bfloat16, "bhtd")


@pytest.mark.gpu
@pytest.mark.parametrize("Tq", [1, 200])
def test_growing_maximum_and_large_scores(Tq):
    """Scores that grow along the keys: the running maximum moves in every tile, by less and by
    more than the step below which the accumulator is left alone."""
    H, Tk, d = 3, 900, 128
    q, k, v, _ = make(1, H, H, Tq, Tk, d, torch.bfloat16, "bhtd", None, sharp=1.0)
    u = torch.randn(d, device="cuda")
    u = u / u.norm()
    ramp = torch.linspace(0, 60, Tk, device="cuda")
    k = (k.float() * 0.3 + ramp[:, None] * u).to(torch.bfloat16)
    q = (q.float() * 0.3 + 12 * u).to(torch.bfloat16)
    cfg = da2.cross_config(1, H, Tq, Tk, d)
    ws = da2.cross_attention_workspace(cfg, "cuda")
    out, lse = torch.empty_like(q), torch.empty(1, H, Tq, device="cuda")
    da2.cross_attention(cfg, q, k, v, out, ws, lse=lse)
    check_out(out, lse, formulas64(q, k, v, None, "bhtd"), torch.bfloat16, "bhtd")


@pytest.mark.gpu
def test_scale_lengths_out_of_range_and_untouched_rows():
    B, H, Tq, Tk, d = 2, 2, 150, 100, 64
    q, k, v, _ = make(B, H, H, Tq, Tk, d, torch.bfloat16, "bthd", None)
    cfg = da2.cross_config(B, H, Tq, Tk, d, sm_scale=0.3, layout="bthd")
    ws = da2.cross_attention_workspace(cfg, "cuda")
    buf = torch.full((B, Tq + 20, H, d), 9.0, dtype=torch.bfloat16, device="cuda")
    lens = [-5, 1000]                                   # taken as 0 and Tk
    da2.cross_attention(cfg, q, k, v, buf[:, :Tq], ws, kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    check_out(buf[:, :Tq], None, formulas64(q, k, v, lens, "bthd", 0.3), torch.bfloat16, "bthd")
    assert (buf[:, Tq:] == 9.0).all() and (buf[0, :Tq] == 0).all()


@pytest.mark.gpu
def test_fused_projection_slices_streams_and_graphs():
    """Keys and values as slices of one projection; another stream; a captured graph replayed
    with other inputs; two calls at once with workspaces of their own."""
    B, H, Tq, Tk, d = 2, 6, 3, 700, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    kv = torch.randn(B, Tk, 2, H, d, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn(B, Tq, H, d, generator=g, device="cuda").to(torch.bfloat16)
    k, v = kv[:, :, 0], kv[:, :, 1]
    cfg = da2.cross_config(B, H, Tq, Tk, d, layout="bthd")
    ws, ws2 = (da2.cross_attention_workspace(cfg, "cuda") for _ in range(2))
    out, out2, lens = torch.empty_like(q), torch.empty_like(q), torch.tensor([700, 333], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    da2.cross_attention(cfg, q, k, v, out, ws, kv_len=lens, stream=s1)
    da2.cross_attention(cfg, q, k, v, out2, ws2, kv_len=lens, stream=s2)
    torch.cuda.synchronize()
    check_out(out, None, formulas64(q, k, v, [700, 333], "bthd"), torch.bfloat16, "bthd")
    assert torch.equal(out, out2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        da2.cross_attention(cfg, q, k, v, out, ws, kv_len=lens)
    q.copy_(torch.randn(q.shape, generator=g, device="cuda"))
    lens.copy_(torch.tensor([0, 512], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    check_out(out, None, formulas64(q, k, v, [0, 512], "bthd"), torch.bfloat16, "bthd")


@pytest.mark.gpu
def test_wait_that_runs_out_is_reported():
    """The test hook withholds the first load; the bounded waits end the call, the error word is
    set, and the next call is right."""
    q, k, v, _ = make(1, 2, 2, 300, 200, 128, torch.bfloat16, "bhtd", None)
    cfg = da2.cross_config(1, 2, 300, 200, 128, flags=da2.FLAG_TEST_STALL)
    ws = da2.cross_attention_workspace(cfg, "cuda")
    out = torch.empty_like(q)
    da2.cross_attention(cfg, q, k, v, out, ws)
    assert da2.cross_attention_get_error(ws) == 1
    assert da2.cross_attention_get_error(ws) == 0
    cfg = da2.cross_config(1, 2, 300, 200, 128)
    da2.cross_attention(cfg, q, k, v, out, ws)
    assert da2.cross_attention_get_error(ws) == 0
    check_out(out, None, formulas64(q, k, v, None, "bhtd"), torch.bfloat16, "bhtd")
