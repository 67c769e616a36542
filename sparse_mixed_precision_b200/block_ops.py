"""Operators of a video-DiT block around the sparse self-attention: the RMS norm and position
rotation of its queries and keys, and the attention of its tokens to an encoder's states, each
with its backward pass (see include/da2.h). Argument marshalling only, like the package's other
calls; the names are re-exported by the package.

    cfg = norm_rope_config(B, Hq, Hk, T, d, layout="bthd")
    qk_norm_rope(cfg, q, k, wq, wk, cos, sin, q_out, k_out)          # then da2.forward(...)

    cfg = cross_config(B, H, Tq, Tk, d)
    ws = cross_attention_workspace(cfg, device)
    cross_attention(cfg, q, k, v, out, ws, kv_len=lens, lse=lse)
    cross_attention_backward(cfg, dout, q, k, v, out, lse, dq, dk, dv, ws_back, kv_len=lens)

Activations are [B, H, T, d] (layout "bhtd") or [B, T, H, d] ("bthd"), bf16 or fp16, with
contiguous channels; the other strides are free (a slice of a fused projection goes in as it
is), multiples of 8 elements. A call runs on the given stream's device, whichever device is
current.
"""
from __future__ import annotations

import contextlib
import ctypes

import sparse_mixed_precision_b200 as _pkg

ROPE_HALVES = 1
ROPE_BATCHED = 2


class Tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("sb", ctypes.c_int64), ("sh", ctypes.c_int64), ("st", ctypes.c_int64)]


class NormRopeConfig(ctypes.Structure):
    """da2_norm_rope_config; `layout` is kept for the binding's shape checks."""
    _fields_ = [(n, ctypes.c_int) for n in ("B", "Hq", "Hk", "T", "d", "T_rot")] + \
               [("eps", ctypes.c_float), ("dtype", ctypes.c_int), ("flags", ctypes.c_int)]
    layout = "bhtd"


class CrossConfig(ctypes.Structure):
    """da2_cross_config; `layout` is kept for the binding's shape checks."""
    _fields_ = [(n, ctypes.c_int) for n in ("B", "H", "Hkv", "Tq", "Tk", "d")] + \
               [("sm_scale", ctypes.c_float), ("dtype", ctypes.c_int), ("flags", ctypes.c_int)]
    layout = "bhtd"


_vp, _sz, _tp = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(Tensor)
_np, _xp, _szp = ctypes.POINTER(NormRopeConfig), ctypes.POINTER(CrossConfig), ctypes.POINTER(ctypes.c_size_t)
SIGNATURES = {
    "da2_qk_norm_rope": [_np, _tp, _tp, _vp, _vp, _vp, _vp, _tp, _tp, _vp],
    "da2_qk_norm_rope_workspace_size": [_np, _szp],
    "da2_qk_norm_rope_backward": [_np, _tp, _tp, _tp, _tp, _vp, _vp, _vp, _vp, _tp, _tp, _vp, _vp, _vp, _sz, _vp],
    "da2_cross_attention_workspace_size": [_xp, _szp],
    "da2_cross_attention": [_xp, _tp, _tp, _tp, _tp, _vp, _vp, _vp, _sz, _vp],
    "da2_cross_attention_backward_workspace_size": [_xp, _szp],
    "da2_cross_attention_backward": [_xp, _tp, _tp, _tp, _tp, _tp, _vp, _vp, _tp, _tp, _tp, _vp, _sz, _vp],
    "da2_cross_attention_get_error": [_vp, _sz, _vp, ctypes.POINTER(ctypes.c_uint32)],
}


_torch = None                       # imported with the first call, like everywhere in the package
_DTYPES = {}                        # DA2_DTYPE_* -> torch dtype


def _load():
    global _torch
    if _torch is None:
        import torch
        _DTYPES.update({0: torch.bfloat16, 1: torch.float16})
        _torch = torch
    return _torch


def _dtype_code(dtype):
    torch = _load()
    dtype = torch.bfloat16 if dtype is None else dtype
    for code, d in _DTYPES.items():
        if d == dtype:
            return code
    raise ValueError(f"dtype must be bfloat16 or float16, not {dtype}")


def _with_layout(cfg, layout):
    if layout not in ("bhtd", "bthd"):
        raise ValueError(f"layout must be 'bhtd' or 'bthd', not {layout!r}")
    cfg.layout = layout
    return cfg


def norm_rope_config(B, Hq, Hk, T, d, dtype=None, T_rot=None, eps=1e-6, layout="bhtd", half=False,
                     batched=False) -> NormRopeConfig:
    """da2_norm_rope_config. dtype: bfloat16 (the default) or float16; T_rot: rotated tokens
    (all of them by default); half: rotate channel pairs (c, c + d/2) instead of (2c, 2c + 1);
    batched: tables [B, T_rot, d/2] instead of [T_rot, d/2]. Hk = 0: queries only."""
    flags = (ROPE_HALVES if half else 0) | (ROPE_BATCHED if batched else 0)
    return _with_layout(NormRopeConfig(B, Hq, Hk, T, d, T if T_rot is None else T_rot, float(eps),
                                       _dtype_code(dtype), flags), layout)


def cross_config(B, H, Tq, Tk, d, Hkv=None, dtype=None, sm_scale=0.0, layout="bhtd", flags=0) -> CrossConfig:
    """da2_cross_config. Hkv: key/value heads (H by default; must divide H); sm_scale: 0 selects
    1/sqrt(d); dtype: bfloat16 (the default) or float16."""
    return _with_layout(CrossConfig(B, H, H if Hkv is None else Hkv, Tq, Tk, d, float(sm_scale),
                                    _dtype_code(dtype), int(flags)), layout)


class _Args:
    """Checks a call's tensors (the C ABI sees bare pointers) and turns them into its arguments.
    Every device tensor must sit on the device of the stream the call runs on."""

    __slots__ = ("fn", "cfg", "dtype", "bthd", "stream", "index")

    def __init__(self, fn, cfg, stream):
        torch = _load()
        self.fn, self.cfg, self.bthd = fn, cfg, cfg.layout == "bthd"
        self.dtype = _DTYPES.get(cfg.dtype)
        if stream is None and torch.cuda.is_initialized():
            stream = torch.cuda.current_stream()
        self.stream = stream
        self.index = -2 if stream is None else stream.device_index

    def _refuse(self, name, t, dtype, shape):
        """The error of a tensor that a check has turned down."""
        if not isinstance(t, _torch.Tensor):
            raise TypeError(f"{self.fn}: {name} must be a torch.Tensor")
        if t.dtype != dtype and dtype is not None:
            raise ValueError(f"{self.fn}: {name} has dtype {t.dtype}; the call needs {dtype}")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{self.fn}: {name} has shape {tuple(t.shape)}; the call needs {tuple(shape)}")
        if t.device.type != "cuda":
            raise ValueError(f"{self.fn}: {name} must be a CUDA tensor, not on {t.device}")
        raise ValueError(f"{self.fn}: {name} is on {t.device} but the call runs on "
                         f"{'no device' if self.stream is None else self.stream.device}")

    def act(self, name, t, H, T):
        """A strided activation of H heads and T tokens."""
        cfg = self.cfg
        want = (cfg.B, T, H, cfg.d) if self.bthd else (cfg.B, H, T, cfg.d)
        if not (isinstance(t, _torch.Tensor) and t.dtype is self.dtype and t.shape == want):
            self._refuse(name, t, self.dtype, want)
        sb, s1, s2, sc = t.stride()
        if sc != 1:
            raise ValueError(f"{self.fn}: {name} must have contiguous channels")
        if t.get_device() != self.index:
            self._refuse(name, t, self.dtype, want)
        return Tensor(t.data_ptr(), sb, s2, s1) if self.bthd else Tensor(t.data_ptr(), sb, s1, s2)

    def plain(self, name, t, dtype, shape):
        """The address of a contiguous tensor of one shape, or None."""
        if t is None:
            return None
        if not (isinstance(t, _torch.Tensor) and t.dtype is dtype and t.shape == shape):
            self._refuse(name, t, dtype, shape)
        if not t.is_contiguous():
            raise ValueError(f"{self.fn}: {name} must be contiguous")
        if t.get_device() != self.index:
            self._refuse(name, t, dtype, shape)
        return t.data_ptr()

    def buffer(self, name, t):
        """A contiguous byte buffer: (address, size)."""
        if not isinstance(t, _torch.Tensor):
            self._refuse(name, t, None, None)
        if not t.is_contiguous():
            raise ValueError(f"{self.fn}: {name} must be contiguous")
        if t.get_device() != self.index:
            self._refuse(name, t, None, None)
        return t.data_ptr(), t.nbytes

    def call(self, *args):
        cuda = _torch.cuda
        here = cuda.current_device() == self.index
        with contextlib.nullcontext() if here else cuda.device(self.index):
            st = getattr(_pkg.lib(), self.fn)(self.cfg, *args, self.stream.cuda_stream)
        if st:
            _pkg._check(self.fn, st)


def _size(fn, cfg):
    n = ctypes.c_size_t()
    _pkg._check(fn, getattr(_pkg.lib(), fn)(ctypes.byref(cfg), ctypes.byref(n)))
    return n.value


def _norm_args(a, cfg, wq, wk, cos, sin):
    f32 = _torch.float32
    table = (cfg.T_rot, cfg.d // 2) if not cfg.flags & ROPE_BATCHED else (cfg.B, cfg.T_rot, cfg.d // 2)
    if cfg.T_rot > 0 and (cos is None or sin is None):
        raise ValueError(f"{a.fn}: cos and sin are needed to rotate {cfg.T_rot} tokens")
    if cfg.T_rot == 0:
        cos = sin = None
    return (a.plain("wq", wq, f32, (cfg.d,)), a.plain("wk", wk, f32, (cfg.d,)),
            a.plain("cos", cos, f32, table), a.plain("sin", sin, f32, table))


def _key_act(a, cfg, name, t):
    return a.act(name, t, cfg.Hk, cfg.T) if cfg.Hk else None


def qk_norm_rope(cfg, q, k, wq, wk, cos, sin, q_out, k_out, stream=None):
    """RMS norm of every head of q and k and the position rotation. wq, wk: float32 [d] or None
    (ones); cos, sin: float32 [T_rot, d/2] ([B, T_rot, d/2] with batched=True); q_out may be q and
    k_out may be k. k and k_out are not used when Hk is 0."""
    a = _Args("da2_qk_norm_rope", cfg, stream)
    a.call(a.act("q", q, cfg.Hq, cfg.T), _key_act(a, cfg, "k", k), *_norm_args(a, cfg, wq, wk, cos, sin),
           a.act("q_out", q_out, cfg.Hq, cfg.T), _key_act(a, cfg, "k_out", k_out))


def qk_norm_rope_workspace_size(cfg) -> int:
    return _size("da2_qk_norm_rope_workspace_size", cfg)


def qk_norm_rope_workspace(cfg, device):
    """A workspace for qk_norm_rope_backward."""
    import torch
    return torch.empty(qk_norm_rope_workspace_size(cfg), dtype=torch.uint8, device=device)


def qk_norm_rope_backward(cfg, dq_out, dk_out, q, k, wq, wk, cos, sin, dq, dk, dwq, dwk, ws, stream=None):
    """Gradients of qk_norm_rope: dq, dk (of q, k) and dwq, dwk (float32 [d], or None) from
    dq_out, dk_out (of its outputs) and its inputs. dq may be dq_out or q, dk may be dk_out or k."""
    a = _Args("da2_qk_norm_rope_backward", cfg, stream)
    f32 = _torch.float32
    dw = a.plain("dwq", dwq, f32, (cfg.d,)), a.plain("dwk", dwk, f32, (cfg.d,))
    a.call(a.act("dq_out", dq_out, cfg.Hq, cfg.T), _key_act(a, cfg, "dk_out", dk_out),
           a.act("q", q, cfg.Hq, cfg.T), _key_act(a, cfg, "k", k), *_norm_args(a, cfg, wq, wk, cos, sin),
           a.act("dq", dq, cfg.Hq, cfg.T), _key_act(a, cfg, "dk", dk), *dw, *a.buffer("ws", ws))


def cross_attention_workspace_size(cfg, backward=False) -> int:
    return _size("da2_cross_attention_backward_workspace_size" if backward else
                 "da2_cross_attention_workspace_size", cfg)


def cross_attention_workspace(cfg, device, backward=False):
    """A workspace for cross_attention (or its backward pass): its error word starts at zero."""
    import torch
    ws = torch.empty(cross_attention_workspace_size(cfg, backward), dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def _cross_args(a, cfg, lse, kv_len):
    return (a.plain("lse", lse, _torch.float32, (cfg.B, cfg.H, cfg.Tq)),
            a.plain("kv_len", kv_len, _torch.int32, (cfg.B,)))


def cross_attention(cfg, q, k, v, out, ws, kv_len=None, lse=None, stream=None):
    """out = softmax(q k^T sm_scale) v over each batch entry's first kv_len[b] keys (int32 [B];
    None: all Tk). lse: float32 [B, H, Tq], or None when no backward pass follows."""
    a = _Args("da2_cross_attention", cfg, stream)
    a.call(a.act("q", q, cfg.H, cfg.Tq), a.act("k", k, cfg.Hkv, cfg.Tk), a.act("v", v, cfg.Hkv, cfg.Tk),
           a.act("out", out, cfg.H, cfg.Tq), *_cross_args(a, cfg, lse, kv_len), *a.buffer("ws", ws))


def cross_attention_backward(cfg, dout, q, k, v, out, lse, dq, dk, dv, ws, kv_len=None, stream=None):
    """Gradients dq, dk, dv of cross_attention from dout, its inputs, its output and its lse. Keys
    and values behind kv_len[b] get zero."""
    a = _Args("da2_cross_attention_backward", cfg, stream)
    if lse is None:
        raise ValueError("da2_cross_attention_backward: lse is needed")
    a.call(a.act("dout", dout, cfg.H, cfg.Tq), a.act("q", q, cfg.H, cfg.Tq), a.act("k", k, cfg.Hkv, cfg.Tk),
           a.act("v", v, cfg.Hkv, cfg.Tk), a.act("out", out, cfg.H, cfg.Tq), *_cross_args(a, cfg, lse, kv_len),
           a.act("dq", dq, cfg.H, cfg.Tq), a.act("dk", dk, cfg.Hkv, cfg.Tk), a.act("dv", dv, cfg.Hkv, cfg.Tk),
           *a.buffer("ws", ws))


def cross_attention_get_error(ws, stream=None) -> int:
    """Reads and clears the error word of a cross_attention workspace (synchronises the stream)."""
    torch = _load()
    if not isinstance(ws, torch.Tensor) or ws.device.type != "cuda":
        raise ValueError("da2_cross_attention_get_error: ws must be a CUDA tensor")
    s = torch.cuda.current_stream(ws.device) if stream is None else stream
    word = ctypes.c_uint32()
    with torch.cuda.device(s.device):
        st = _pkg.lib().da2_cross_attention_get_error(ctypes.c_void_p(ws.data_ptr()), ws.numel() * ws.element_size(),
                                                      ctypes.c_void_p(s.cuda_stream), ctypes.byref(word))
    if st not in (0, 6):
        raise _pkg.DA2Error("da2_cross_attention_get_error", st)
    return word.value
