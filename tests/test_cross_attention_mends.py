"""Attention to an encoder's states at the places where it once went wrong: short keys over many query
tiles, gradients over fp16's range, long batches, parts without weight, aborted calls."""
import pytest
import torch

import sparse_mixed_precision_b200 as da2
from tests.test_cross_attention import check_out, formulas64, make
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


# ------------------------------------------------------------------ gradients over fp16's range
def fp16_wants(q, k, v, dout, lens):
    """gradients64 plus what dS may lose below fp16's smallest normal. dS is rounded with a power of two
    of at least 2^13 / bound, bound = max |dout row| max |v row| over the query heads of a key/value
    head, so that a subnormal is off by at most 2^-25 2^-13 bound."""
    want = gradients64(q, k, v, dout, lens, "bhtd", torch.float16)
    B, H, Tq, d = q.shape
    Hkv = k.shape[1]
    for b in range(B):
        n = k.shape[2] if lens is None else lens[b]
        if n == 0:
            continue
        rows = dout[b].double().norm(dim=-1).view(Hkv, -1).amax(-1)
        tiny = (rows * v[b, :, :n].double().norm(dim=-1).amax(-1) * 2.0 ** -38 / d ** 0.5)[:, None, None]
        want[0][1][b] += (tiny * k[b, :, :n].double().abs().sum(1, keepdim=True)).repeat_interleave(H // Hkv, 0)
        want[1][1][b, :, :n] += tiny * q[b].double().abs().view(Hkv, -1, d).sum(1, keepdim=True)
    return want


FP16_CASES = [  # B, H, Hkv, Tq, Tk, d, lens
    (1, 2, 2, 200, 16, 128, None), (2, 4, 2, 130, 77, 128, [77, 5]), (1, 2, 1, 300, 512, 128, None),
    (2, 2, 2, 150, 300, 64, [300, 129]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", FP16_CASES)
@pytest.mark.parametrize("scale", [2.0 ** 9, 300.0, 2.0 ** -9, 2.0 ** -14])
def test_fp16_gradients_of_large_and_small_dout(case, scale):
    """|dS| far above 1023 and far below fp16's normals, as loss scaling leaves them: the gradients are
    ordinary fp16 numbers throughout."""
    B, H, Hkv, Tq, Tk, d, lens = case
    q, k, v, kv_len = make(B, H, Hkv, Tq, Tk, d, torch.float16, "bhtd", lens)
    g = torch.Generator(device="cuda").manual_seed(9)
    dout = (torch.randn(q.shape, generator=g, device="cuda") * scale).half()
    cfg = da2.cross_config(B, H, Tq, Tk, d, Hkv=Hkv, dtype=torch.float16)
    _, _, grads = run_both(cfg, q, k, v, dout, kv_len)
    want = fp16_wants(q, k, v, dout, lens)
    assert all(x.abs().max() < 65504 for x, _ in want)
    check_grads(grads, want, "bhtd")


@pytest.mark.gpu
@pytest.mark.parametrize("case", FP16_CASES)
def test_fp16_gradients_of_uneven_rows(case):
    """One row of dout 2^8 and one value row 2^3 times the others."""
    B, H, Hkv, Tq, Tk, d, lens = case
    q, k, v, kv_len = make(B, H, Hkv, Tq, Tk, d, torch.float16, "bhtd", lens, seed=5)
    dout = torch.randn(q.shape, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").half()
    dout[:, 0, 70] *= 2.0 ** 8
    v[:, :, 3] *= 2.0 ** 3
    cfg = da2.cross_config(B, H, Tq, Tk, d, Hkv=Hkv, dtype=torch.float16)
    _, _, grads = run_both(cfg, q, k, v, dout, kv_len)
    check_grads(grads, fp16_wants(q, k, v, dout, lens), "bhtd")


@pytest.mark.gpu
@pytest.mark.parametrize("Tk", [90, 300])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_fp16_infinite_gradient_stays_where_it_belongs(Tk, bad):
    """An overflowed element of dout, as loss scaling meets them: its row of dq and its head's dk and
    dv say so, every other row of dq and the other head are as without it."""
    q, k, v, _ = make(1, 2, 2, 260, Tk, 128, torch.float16, "bhtd", None, seed=6)
    dout = torch.randn(q.shape, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").half()
    cfg = da2.cross_config(1, 2, 260, Tk, 128, dtype=torch.float16)
    out, lse, clean = run_both(cfg, q, k, v, dout, None)
    dout[0, 0, 150, 7] = bad
    dq, dk, dv = (torch.empty_like(x) for x in clean)
    ws = da2.cross_attention_workspace(cfg, "cuda", backward=True)
    da2.cross_attention_backward(cfg, dout, q, k, v, out, lse, dq, dk, dv, ws)
    assert not torch.isfinite(dq[0, 0, 150]).any() and not torch.isfinite(dk[0, 0]).any()
    assert not torch.isfinite(dv[0, 0, :, 7]).any()
    keep = torch.arange(260, device="cuda") != 150
    assert torch.equal(dq[0, 0, keep], clean[0][0, 0, keep]) and torch.equal(dv[0, 0, :, 8:], clean[2][0, 0, :, 8:])
    assert all(torch.equal(a[0, 1], b[0, 1]) for a, b in zip((dq, dk, dv), clean))


@pytest.mark.gpu
def test_fp16_gradients_captured():
    """The fp16 backward pass, whose kernels overlap, captured and replayed with other values, sizes of
    dout and lengths; the workspace's norms are those of the replay."""
    B, H, Tq, Tk, d = 2, 3, 400, 300, 128
    q, k, v, _ = make(B, H, H, Tq, Tk, d, torch.float16, "bhtd", None, seed=8)
    gen = torch.Generator(device="cuda").manual_seed(4)
    dout = torch.randn(q.shape, generator=gen, device="cuda").half()
    lens = torch.tensor([300, 140], dtype=torch.int32, device="cuda")
    cfg = da2.cross_config(B, H, Tq, Tk, d, dtype=torch.float16)
    out, lse, first = run_both(cfg, q, k, v, dout, lens)
    ws, wsb = da2.cross_attention_workspace(cfg, "cuda"), da2.cross_attention_workspace(cfg, "cuda", backward=True)
    grads = [torch.empty_like(x) for x in first]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        da2.cross_attention(cfg, q, k, v, out, ws, kv_len=lens, lse=lse)
        da2.cross_attention_backward(cfg, dout, q, k, v, out, lse, *grads, wsb, kv_len=lens)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, grads))
    v.mul_(16.0)
    dout.mul_(64.0)
    for n in ([0, 257], [128, 300]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        for _ in range(3):
            graph.replay()
        check_grads(grads, fp16_wants(q, k, v, dout, n), "bhtd")


# ------------------------------------------------------------------ long batches
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_many_short_sequences_with_lengths_of_their_own(dtype):
    """Hundreds of batch entries, some without a key, some with several key tiles."""
    B, H, Hkv, Tq, Tk, d = 333, 4, 2, 9, 150, 64
    gen = torch.Generator().manual_seed(7)
    lens = [int(n) for n in torch.randint(-40, Tk + 1, (B,), generator=gen).clamp(min=0)]
    q, k, v, kv_len = make(B, H, Hkv, Tq, Tk, d, dtype, "bhtd", lens, seed=2)
    dout = torch.randn(q.shape, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(dtype)
    cfg = da2.cross_config(B, H, Tq, Tk, d, Hkv=Hkv, dtype=dtype)
    _, _, grads = run_both(cfg, q, k, v, dout, kv_len)
    check_grads(grads, gradients64(q, k, v, dout, lens, "bhtd", dtype), "bhtd")


@pytest.mark.gpu
def test_backward_time_grows_with_the_batch_and_not_its_square():
    """Frames or windows folded into the batch: eight times the entries may take twice as long an entry,
    not eight times."""
    H, T, d = 8, 8, 64

    def time_of(B):
        x = torch.randn(B, H, T, d, device="cuda").to(torch.bfloat16)
        lse = torch.zeros(B, H, T, device="cuda")
        lens = torch.full((B,), T, dtype=torch.int32, device="cuda")
        cfg = da2.cross_config(B, H, T, T, d)
        ws = da2.cross_attention_workspace(cfg, "cuda", backward=True)
        grads = [torch.empty_like(x) for _ in range(3)]
        best = float("inf")
        for _ in range(4):
            t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            t[0].record()
            da2.cross_attention_backward(cfg, x, x, x, x, x, lse, *grads, ws, kv_len=lens)
            t[1].record()
            t[1].synchronize()
            best = min(best, t[0].elapsed_time(t[1]))
        assert da2.cross_attention_get_error(ws) == 0
        return best

    short, long = time_of(2048), time_of(16384)
    assert long <= 16 * short, (short, long)


# ------------------------------------------------------------------ parts without weight
@pytest.mark.gpu
@pytest.mark.parametrize("Tq", [1, 300])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_keys_of_infinitely_low_score(Tq, dtype):
    """Keys whose score is -inf, as a channel used for masking gives them: no weight, also where they fill
    a whole part of the split keys; with no other key the softmax has no value."""
    H, Tk, d = 2, 4096, 64
    q, k, v, _ = make(2, H, H, Tq, Tk, d, dtype, "bhtd", None, seed=4)
    q[..., 0] = 1
    k[0, 0, :, 0] = torch.where(torch.arange(Tk, device="cuda") < 3900, -float("inf"), 0.0)
    k[0, 1, 100:, 0] = -float("inf")
    k[1, 1, :, 0] = -float("inf")
    cfg = da2.cross_config(2, H, Tq, Tk, d, dtype=dtype)
    ws = da2.cross_attention_workspace(cfg, "cuda")
    assert ws.numel() > 256                             # the keys are split
    out, lse = torch.empty_like(q), torch.empty(2, H, Tq, device="cuda")
    da2.cross_attention(cfg, q, k, v, out, ws, lse=lse)
    for b, h in ((0, 0), (0, 1), (1, 0)):
        at = (slice(b, b + 1), slice(h, h + 1))
        keys = {(0, 0): slice(3900, None), (0, 1): slice(0, 100), (1, 0): slice(None)}[b, h]
        check_out(out[at], lse[at], formulas64(q[at], k[at][:, :, keys], v[at][:, :, keys], None, "bhtd"), dtype, "bhtd")
    assert torch.isnan(out[1, 1]).all() and (lse[1, 1] == -float("inf")).all()


@pytest.mark.gpu
@pytest.mark.parametrize("Tk", [64, 4096])
def test_a_nan_query_has_a_nan_row(Tk):
    """With one part and with several: the row and its lse are NaN, the other rows are as without it."""
    q, k, v, _ = make(1, 2, 2, 3, Tk, 128, torch.bfloat16, "bhtd", None, seed=4)
    cfg = da2.cross_config(1, 2, 3, Tk, 128)
    ws = da2.cross_attention_workspace(cfg, "cuda")
    assert (ws.numel() > 256) == (Tk == 4096)
    out, clean, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(1, 2, 3, device="cuda")
    da2.cross_attention(cfg, q, k, v, clean, ws, lse=lse)
    q[0, 1, 1, 5] = float("nan")
    da2.cross_attention(cfg, q, k, v, out, ws, lse=lse)
    assert torch.isnan(out[0, 1, 1]).all() and torch.isnan(lse[0, 1, 1])
    out[0, 1, 1] = clean[0, 1, 1]
    assert torch.equal(out, clean) and torch.isnan(lse).sum() == 1


# ------------------------------------------------------------------ calls that are given up
@pytest.mark.gpu
def test_an_aborted_call_ends_soon_after_the_limit():
    """The test hook withholds each kernel's first load and its waits run out. What a long call then takes
    beyond a short one, whose waits are few, is about its arithmetic (35 ms here), not the number of its
    waits times their suspension."""
    def stalled(H, Tq, Tk):
        x = torch.zeros(1, H, Tq, 128, dtype=torch.bfloat16, device="cuda")
        k, lse = x[:, :, :Tk].contiguous(), torch.zeros(1, H, Tq, device="cuda")
        grads = [torch.empty_like(t) for t in (x, k, k)]
        cfg = da2.cross_config(1, H, Tq, Tk, 128, flags=da2.FLAG_TEST_STALL)
        ws = da2.cross_attention_workspace(cfg, "cuda", backward=True)
        t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        t[0].record()
        da2.cross_attention_backward(cfg, x, x, k, k, x, lse, *grads, ws)
        t[1].record()
        t[1].synchronize()
        assert da2.cross_attention_get_error(ws) == 1
        return t[0].elapsed_time(t[1])

    stalled(2, 4096, 4096)                              # loads the kernels
    short, long = stalled(2, 4096, 4096), stalled(40, 131072, 4096)
    assert long - short < 45, (short, long)
