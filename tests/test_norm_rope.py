"""The norm and rotation of queries and keys: refusals (host checks, no CUDA call) and, on a GPU,
both directions against the formulas in 64 bits and the gradients against differences."""
import ctypes

import pytest
import torch

import sparse_mixed_precision_b200 as da2

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ refusals, no GPU
def _status(cfg, q="ok", cos=0x1000, strides=None, fn="da2_qk_norm_rope"):
    """Status of a call whose pointers are never read: every refusal comes before the launch."""
    from sparse_mixed_precision_b200.block_ops import Tensor
    B, H, T, d = cfg.B, max(cfg.Hq, 1), cfg.T, cfg.d
    good = Tensor(0x1000, H * T * d, T * d, d)
    bad = {"ok": good, "null": Tensor(None, H * T * d, T * d, d), "odd": Tensor(0x1008, H * T * d, T * d, d)}[q]
    if strides:
        bad = Tensor(0x1000, *strides)
    t, g = ctypes.byref(bad), ctypes.byref(good)
    L = da2.lib()
    if fn == "da2_qk_norm_rope":
        return L.da2_qk_norm_rope(ctypes.byref(cfg), t, g, None, None, cos, cos, g, g, None)
    return L.da2_qk_norm_rope_backward(ctypes.byref(cfg), t, g, g, g, None, None, cos, cos, g, g, 0x1000, 0x1000,
                                       0x1000, 16, None)


def _cfg(**kw):
    base = dict(B=2, Hq=3, Hk=3, T=10, d=64)
    base.update(kw)
    return da2.norm_rope_config(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(Hq=0), 1), (dict(Hk=-1), 1), (dict(T=0), 1), (dict(T_rot=11), 1), (dict(T_rot=-1), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("inf")), 1), (dict(eps=float("nan")), 1), (dict(d=96), 2), (dict(d=256), 2),
    (dict(B=1 << 20, T=1 << 20), 2),
])
def test_bad_configurations_are_refused(kw, status):
    assert _status(_cfg(**kw)) == status
    n = ctypes.c_size_t()
    assert da2.lib().da2_qk_norm_rope_workspace_size(ctypes.byref(_cfg(**kw)), ctypes.byref(n)) == status


def test_bad_arguments_are_refused():
    assert _status(_cfg(), q="null") == 1
    assert _status(_cfg(), q="odd") == 3
    assert _status(_cfg(), cos=None) == 1
    assert _status(_cfg(), cos=0x1004) == 3
    assert _status(_cfg(), strides=(0, 640, 64)) == 1          # broadcast batch
    assert _status(_cfg(), strides=(1920, -640, 64)) == 1
    assert _status(_cfg(), strides=(1920, 640, 32)) == 1       # rows would overlap
    assert _status(_cfg(), strides=(1920, 640, 68)) == 3       # token stride not a multiple of 8
    c = _cfg()
    c.flags = 4
    assert _status(c) == 1
    c = _cfg()
    c.dtype = 7
    assert _status(c) == 1
    assert _status(_cfg(), fn="back") == 4                     # 16 bytes of workspace
    assert da2.lib().da2_qk_norm_rope(None, None, None, None, None, None, None, None, None, None) == 1


def test_binding_checks_tensors():
    cfg = _cfg()
    x = torch.zeros(2, 3, 10, 64, dtype=torch.bfloat16)
    cs = torch.zeros(10, 32)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        da2.qk_norm_rope(cfg, x, x, None, None, cs, cs, x, x)
    with pytest.raises(ValueError, match="dtype"):
        da2.qk_norm_rope(cfg, x.half(), x, None, None, cs, cs, x, x)
    with pytest.raises(ValueError, match="shape"):
        da2.qk_norm_rope(cfg, x[:, :2], x, None, None, cs, cs, x, x)
    with pytest.raises(ValueError, match="contiguous channels"):
        da2.qk_norm_rope(cfg, torch.zeros(2, 3, 10, 128, dtype=torch.bfloat16)[..., ::2], x, None, None, cs, cs, x, x)
    with pytest.raises(TypeError):
        da2.qk_norm_rope(cfg, None, x, None, None, cs, cs, x, x)
    with pytest.raises(ValueError, match="dtype"):
        da2.norm_rope_config(1, 1, 1, 1, 64, dtype=torch.float32)
    with pytest.raises(ValueError, match="layout"):
        da2.norm_rope_config(1, 1, 1, 1, 64, layout="tbhd")


# ------------------------------------------------------------------ GPU
def _rotate64(x, cos, sin, half, sign=1):
    """x [B, H, T, d] float64; cos, sin [B or 1, T_rot, d/2]."""
    n, d = cos.shape[-2], x.shape[-1]
    a_ix, b_ix = (slice(0, d // 2), slice(d // 2, d)) if half else (slice(0, d, 2), slice(1, d, 2))
    y = x.clone()
    c, s = cos.double()[:, None], sign * sin.double()[:, None]
    a, b = x[:, :, :n, a_ix], x[:, :, :n, b_ix]
    y[:, :, :n, a_ix] = a * c - b * s
    y[:, :, :n, b_ix] = a * s + b * c
    return y


def _forward64(x, w, cos, sin, half, eps):
    x = x.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return _rotate64(y if w is None else y * w.double(), cos, sin, half)


def _make(B, Hq, Hk, T, d, dt, layout, T_rot, batched=False, seed=0, wide=False):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def act(H, scale):
        shape = (B, T, H, d) if layout == "bthd" else (B, H, T, d)
        if wide:       # a slice of a wider buffer: strides that no contiguous tensor has
            x = torch.randn(shape[:2] + (shape[2] + 3, d + 16), generator=g, device="cuda") * scale
            return x.to(dt)[:, :, 1:-2, 8:-8]
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dt)

    q, k = act(Hq, 2.0), act(Hk, 0.3) if Hk else None
    wq = 1 + 0.3 * torch.randn(d, generator=g, device="cuda")
    wk = 1 + 0.3 * torch.randn(d, generator=g, device="cuda")
    ang = torch.rand((B if batched else 1, T_rot, d // 2), generator=g, device="cuda", dtype=torch.float64) * 6.3
    cos, sin = ang.cos().float(), ang.sin().float()
    if not batched:
        cos, sin = cos[0], sin[0]
    return q, k, wq, wk, cos, sin


def _heads(x, layout):
    return x.transpose(1, 2) if layout == "bthd" else x


def _close(got, want, dt, extra=0.0):
    """One rounding to dt, half a step relative to the value (plus dt's smallest step), on top of
    fp32 arithmetic: norm, weight and rotation take about 20 roundings of 2^-24 relative to the
    pair's length, covered by 2^-18 of the row's largest value (plus `extra` of it)."""
    row = want.abs().amax(-1, keepdim=True)
    tol = want.abs() * torch.finfo(dt).eps / 2 + row * (2.0 ** -18 + extra) + torch.finfo(dt).smallest_normal
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (bad.sum().item(), (got.double() - want).abs().max().item())


SHAPES = [  # B, Hq, Hk, T, d, T_rot
    (1, 1, 1, 1, 64, 1), (1, 2, 2, 2048, 64, 2048), (2, 3, 1, 33, 128, 20), (1, 40, 40, 65, 128, 65),
    (3, 5, 0, 31, 64, 0), (2, 9, 2, 1001, 128, 924), (1, 1, 24, 7, 64, 7),
]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("layout", ["bhtd", "bthd"])
@pytest.mark.parametrize("half", [False, True])
def test_forward_and_backward_match_the_formulas(shape, dtype, layout, half):
    B, Hq, Hk, T, d, T_rot = shape
    dt = DT[dtype]
    q, k, wq, wk, cos, sin = _make(B, Hq, Hk, T, d, dt, layout, T_rot, wide=T % 2 == 1)
    cfg = da2.norm_rope_config(B, Hq, Hk, T, d, dtype=dt, T_rot=T_rot, eps=1e-5, layout=layout, half=half)
    sides = [("q", q, wq)] + ([("k", k, wk)] if Hk else [])
    oq, ok = torch.empty_like(q), torch.empty_like(k) if Hk else None
    da2.qk_norm_rope(cfg, q, k, wq, wk, cos, sin, oq, ok)
    c3, s3 = (t.reshape(1, T_rot, d // 2) for t in (cos, sin))
    for (name, x, w), o in zip(sides, (oq, ok)):
        _close(_heads(o, layout), _forward64(_heads(x, layout), w, c3, s3, half, 1e-5), dt)

    g = torch.Generator(device="cuda").manual_seed(5)
    dys = [torch.randn(x.shape, generator=g, device="cuda").to(dt) for _, x, _ in sides] + [None]
    dq, dk = torch.empty_like(q), torch.empty_like(k) if Hk else None
    dwq, dwk = torch.full((d,), 7.0, device="cuda"), torch.full((d,), 7.0, device="cuda")
    ws = da2.qk_norm_rope_workspace(cfg, "cuda")
    args = (cfg, dys[0], dys[1], q, k, wq, wk, cos, sin, dq, dk, dwq, dwk, ws)
    da2.qk_norm_rope_backward(*args)
    for (name, x, w), dy, dx, dw in zip(sides, dys, (dq, dk), (dwq, dwk)):
        x64 = _heads(x, layout).double().requires_grad_()
        w64 = w.double().requires_grad_()
        y = _forward64(x64, w64, c3, s3, half, 1e-5)
        gx, gw = torch.autograd.grad(y, (x64, w64), _heads(dy, layout).double())
        _close(_heads(dx, layout), gx, dt, extra=2.0 ** -18)
        # fp32 sums in chains of at most T Hq B / (rows of a block x blocks) + 100 terms, each
        # rounding 2^-24 of a partial sum that stays below the sum of absolute terms
        n = x.double() / torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + 1e-5)
        gr = _rotate64(_heads(dy, layout).double(), c3, s3, half, -1)
        total = (gr * _heads(n, layout)).abs().sum((0, 1, 2))
        assert ((dw.double() - gw).abs() <= total * 2.0 ** -24 * 300).all()
    if not Hk:
        assert (dwk == 7.0).all()
    first = [t.clone() for t in (dq, dwq)]
    da2.qk_norm_rope_backward(*args)
    assert all(torch.equal(a, b) for a, b in zip(first, (dq, dwq)))      # fixed order of the sums


@pytest.mark.gpu
def test_gradients_match_differences():
    """Central differences of the 64-bit formula in a few directions, against the kernel's fp16
    gradient: off by half a step of each element, and the difference quotient's own h^2 error."""
    torch.manual_seed(3)
    B, H, T, d = 1, 2, 5, 64
    q, k, wq, wk, cos, sin = _make(B, H, H, T, d, torch.float16, "bhtd", T)
    cfg = da2.norm_rope_config(B, H, H, T, d, dtype=torch.float16)
    dy = torch.randn_like(q)
    dq, dk, dwq = torch.empty_like(q), torch.empty_like(k), torch.empty_like(wq)
    da2.qk_norm_rope_backward(cfg, dy, dy, q, k, wq, wk, cos, sin, dq, dk, dwq, None, da2.qk_norm_rope_workspace(cfg, "cuda"))
    f = lambda x, w: (_forward64(x, w, cos[None], sin[None], False, 1e-6) * dy.double()).sum()  # noqa: E731
    for _ in range(4):
        u, h = torch.randn(q.shape, device="cuda", dtype=torch.float64), 1e-4
        num = (f(q.double() + h * u, wq) - f(q.double() - h * u, wq)) / (2 * h)
        off = (dq.double().abs() * u.abs()).sum() * 2.0 ** -11 + (u.abs().sum() * 2.0 ** -25)
        assert (num - (dq.double() * u).sum()).abs() <= off + 1e-5 * num.abs() + 1e-6
        u = torch.randn(d, device="cuda", dtype=torch.float64)
        num = (f(q, wq.double() + h * u) - f(q, wq.double() - h * u)) / (2 * h)
        assert (num - (dwq.double() * u).sum()).abs() <= 1e-4 * (dwq.double() * u).abs().sum()


@pytest.mark.gpu
def test_in_place_batched_tables_streams_and_graphs():
    B, H, T, d = 2, 4, 77, 128
    q, k, wq, wk, cos, sin = _make(B, H, H, T, d, torch.bfloat16, "bthd", 70, batched=True)
    cfg = da2.norm_rope_config(B, H, H, T, d, T_rot=70, layout="bthd", batched=True)
    oq, ok = torch.empty_like(q), torch.empty_like(k)
    da2.qk_norm_rope(cfg, q, k, wq, wk, cos, sin, oq, ok)
    _close(oq.transpose(1, 2), _forward64(q.transpose(1, 2), wq, cos, sin, False, 1e-6), torch.bfloat16)
    # in place, on another stream, and captured
    side = torch.cuda.Stream()
    q2, k2 = q.clone(), k.clone()
    torch.cuda.synchronize()
    da2.qk_norm_rope(cfg, q2, k2, wq, wk, cos, sin, q2, k2, stream=side)
    side.synchronize()
    assert torch.equal(q2, oq) and torch.equal(k2, ok)
    ws = da2.qk_norm_rope_workspace(cfg, "cuda")
    dq, dk, dw = torch.empty_like(q), torch.empty_like(k), torch.empty(2, d, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        da2.qk_norm_rope(cfg, q, k, wq, wk, cos, sin, q2, k2)
        da2.qk_norm_rope_backward(cfg, q2, k2, q, k, wq, wk, cos, sin, dq, dk, dw[0], dw[1], ws)
    q2.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q2, oq)
    want = [torch.empty_like(t) for t in (dq, dk, dw)]
    da2.qk_norm_rope_backward(cfg, oq, ok, q, k, wq, wk, cos, sin, want[0], want[1], want[2][0], want[2][1], ws)
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dw), want))
    # gradients in place of the incoming ones
    g1, g2 = oq.clone(), ok.clone()
    da2.qk_norm_rope_backward(cfg, g1, g2, q, k, wq, wk, cos, sin, g1, g2, dw[0], None, ws)
    assert torch.equal(g1, want[0]) and torch.equal(g2, want[1])


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """The last rows of a tensor of more than 2^31 elements."""
    H, d, T = 40, 128, 450000
    q = torch.empty(1, T, H, d, dtype=torch.bfloat16, device="cuda")
    q[:, -3:] = torch.randn(1, 3, H, d, device="cuda").to(torch.bfloat16)
    q[:, :3] = 1
    cfg = da2.norm_rope_config(1, H, 0, T, d, T_rot=0, layout="bthd")
    want = _forward64(q[:, -3:].transpose(1, 2), None, torch.ones(1, 0, 64, device="cuda"),
                      torch.ones(1, 0, 64, device="cuda"), False, 1e-6)
    da2.qk_norm_rope(cfg, q, None, None, None, None, None, q, None)
    _close(q[:, -3:].transpose(1, 2), want, torch.bfloat16)


@pytest.mark.gpu
def test_row_behind_the_tokens_stays():
    """A call on the first tokens of a longer buffer leaves the rest as it was."""
    buf = torch.full((1, 50, 3, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(1, 45, 3, 64, device="cuda").to(torch.bfloat16)
    cfg = da2.norm_rope_config(1, 3, 3, 45, 64, T_rot=0, layout="bthd")
    buf2 = buf.clone()
    da2.qk_norm_rope(cfg, x, x, None, None, None, None, buf[:, :45], buf2[:, :45])
    assert (buf[:, 45:] == 9.0).all() and torch.equal(buf, buf2) and not (buf[:, :45] == 9.0).all()
