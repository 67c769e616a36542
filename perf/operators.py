"""The cases on which the operators around the sparse self-attention are measured.

Two operators, each in both directions, as a video DiT block runs them next to the library's
self-attention:

  norm_rope       RMS norm of every head of the queries and keys and the position rotation, in
                  one pass, in front of da2_prepare; its backward pass gives the gradients of
                  the queries, the keys and the two norm weights.
  cross           attention of the video tokens to an encoder's states (text, image) of another
                  length, with one valid length per batch entry; its backward pass gives the
                  gradients of queries, keys and values.

`run` computes a case with elementary torch operations in 32 bits (own = False), or with the
library's calls (own = True). Sizes come from the library's own workloads (tiny, 480p, 720p and
129-frame layers) and generic encoder lengths.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _norm(name, op, B, Hq, Hk, T, T_rot, d, dtype, layout, style):
    return dict(name=name, op=op, B=B, Hq=Hq, Hk=Hk, T=T, T_rot=T_rot, d=d, dtype=dtype, layout=layout,
                style=style)


def _cross(name, op, B, H, Hkv, Tq, Tk, d, dtype, layout, lens, lse):
    return dict(name=name, op=op, B=B, H=H, Hkv=Hkv, Tq=Tq, Tk=Tk, d=d, dtype=dtype, layout=layout, lens=lens,
                lse=lse)


def listed():
    return [
        # the tiny workload's layer: a call where latency counts
        _norm("norm_tiny", "norm", 1, 2, 2, 2048, 2048, 64, "bf16", "bhtd", "pairs"),
        # the 480p layer as a fused projection leaves it, token-major
        _norm("norm_480p", "norm", 1, 40, 40, 32760, 32760, 128, "bf16", "bthd", "pairs"),
        # the 720p layer, head-major
        _norm("norm_720p", "norm", 1, 40, 40, 75600, 75600, 128, "bf16", "bhtd", "pairs"),
        # fine-tuning on a short odd clip with text tokens behind the video tokens, not rotated
        _norm("norm_back_odd", "norm_back", 2, 3, 3, 1001, 924, 64, "f16", "bthd", "halves"),
        # fine-tuning the 480p layer
        _norm("norm_back_480p", "norm_back", 1, 40, 40, 32760, 32760, 128, "bf16", "bthd", "pairs"),
        # the tiny workload's queries on a short prompt
        _cross("cross_tiny", "cross", 1, 2, 2, 2048, 77, 64, "bf16", "bhtd", "full", False),
        # the 480p layer on a text encoder's 512 states, forward of a training step
        _cross("cross_480p", "cross", 1, 40, 40, 32760, 512, 128, "bf16", "bthd", "full", True),
        # the 720p layer on 512 states, sampling
        _cross("cross_720p", "cross", 1, 40, 40, 75600, 512, 128, "bf16", "bhtd", "full", False),
        # the 129-frame layer, both guidance branches with prompts of their own lengths
        _cross("cross_129f", "cross", 2, 24, 24, 118800, 256, 128, "bf16", "bthd", "ragged", False),
        # one query token a head on a long memory
        _cross("cross_one", "cross", 2, 40, 40, 1, 4096, 128, "bf16", "bthd", "full", False),
        # gradients of a short odd clip on two prompts of different lengths
        _cross("cross_back_odd", "cross_back", 2, 24, 24, 1001, 333, 128, "f16", "bhtd", "ragged", True),
        # gradients of the 480p layer
        _cross("cross_back_480p", "cross_back", 1, 40, 40, 32760, 512, 128, "bf16", "bthd", "full", True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "cross", "cross", "cross_back", "cross_back"])
    B, d = rng.choice([1, 1, 2, 3]), rng.choice([64, 128, 128])
    dtype, layout = rng.choice(["bf16", "bf16", "f16"]), rng.choice(["bhtd", "bthd"])
    H, group = rng.choice([(2, 1), (3, 1), (5, 1), (8, 1), (8, 4), (24, 1), (40, 1), (40, 5)])
    if op.startswith("norm"):
        T = _log_int(rng, 1, 32760 * 40 // (B * H))
        T = min(T, 118800)
        T_rot = T if rng.random() < 0.6 else rng.randint(0, T)
        c = _norm("", op, B, H, H // group, T, T_rot, d, dtype, layout, rng.choice(["pairs", "halves"]))
    else:
        Tk = _log_int(rng, 1, 4500)
        rows = 40 * 32760 * (2 if op == "cross_back" else 4)
        Tq = _log_int(rng, 1, max(1, min(118800, rows // (B * H), 40 * 32760 * 512 // (B * H * Tk))))
        c = _cross("", op, B, H, H // group, Tq, Tk, d, dtype, layout, rng.choice(["full", "ragged"]),
                   op == "cross_back" or rng.random() < 0.5)
    c.pop("name")
    return c


def _lens(case):
    """Valid keys of every batch entry: all of them, or prompts of lengths of their own."""
    B, Tk = case["B"], case["Tk"]
    if case["lens"] == "full":
        return [Tk] * B
    return [max(1, (Tk * (5 + 3 * b) // 7) % (Tk + 1)) for b in range(B)]


def _shape(case, H, T):
    return (case["B"], T, H, case["d"]) if case["layout"] == "bthd" else (case["B"], H, T, case["d"])


def _heads(case, x):
    """[B, H, T, d] view of an activation."""
    return x.transpose(1, 2) if case["layout"] == "bthd" else x


def _rope_tables(T, d, device):
    """cos and sin [T, d/2] of a video's three axes: the tokens are those of frames of 30 x 52
    positions, the channel pairs are shared out among frame, row and column."""
    t = torch.arange(T, device=device)
    axes = (t // (30 * 52), t // 52 % 30, t % 52)
    n = d // 2
    parts = (n - 2 * (n // 3), n // 3, n // 3)
    ang = torch.cat([a.double()[:, None] * (10000.0 ** (-torch.arange(p, device=device).double() / p))[None]
                     for a, p in zip(axes, parts)], 1)
    return ang.cos().float(), ang.sin().float()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt, d = DTYPES[case["dtype"]], case["d"]

    def normal(H, T, scale=1.0):
        x = torch.randn(_shape(case, H, T), generator=gen, device=dev, dtype=torch.float32)
        return (x * scale).to(dt)

    st = {"case": case}
    if case["op"].startswith("norm"):
        Hq, Hk, T = case["Hq"], case["Hk"], case["T"]
        st["q"], st["k"] = normal(Hq, T, 1.7), normal(Hk, T, 0.6)
        st["wq"] = 1.0 + 0.2 * torch.randn(d, generator=gen, device=dev)
        st["wk"] = 1.0 + 0.2 * torch.randn(d, generator=gen, device=dev)
        st["cos"], st["sin"] = _rope_tables(case["T_rot"], d, dev)
        st["eps"] = 1e-6
        st["oq"], st["ok"] = torch.empty_like(st["q"]), torch.empty_like(st["k"])
        if case["op"] == "norm_back":
            st["dq"], st["dk"] = normal(Hq, T, 0.01), normal(Hk, T, 0.01)
            st["dwq"], st["dwk"] = torch.empty_like(st["wq"]), torch.empty_like(st["wk"])
    else:
        H, Hkv, Tq, Tk = case["H"], case["Hkv"], case["Tq"], case["Tk"]
        # normed queries and keys: scores of about unit variance, some heads sharper
        st["q"], st["k"], st["v"] = normal(H, Tq, 1.5), normal(Hkv, Tk), normal(Hkv, Tk)
        st["len"] = torch.tensor(_lens(case), dtype=torch.int32, device=dev)
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty((case["B"], H, Tq), dtype=torch.float32, device=dev) if case["lse"] else None
        if case["op"] == "cross_back":
            o, lse = _cross_plain(case, st)
            st["out"].copy_(o)
            st["lse"].copy_(lse)
            del o, lse
            st["dout"] = normal(H, Tq, 0.01)
            st["dq"], st["dk"], st["dv"] = (torch.empty_like(st[n]) for n in ("q", "k", "v"))
    return st


def _rotate(case, y, cos, sin):
    """Rotates the first T_rot tokens of y [B, H, T, d] by the tables."""
    n, h = case["T_rot"], case["d"] // 2
    r = y[:, :, :n]
    out = y.clone()
    if case["style"] == "pairs":
        a, b = r[..., 0::2], r[..., 1::2]
        out[:, :, :n, 0::2] = a * cos - b * sin
        out[:, :, :n, 1::2] = a * sin + b * cos
    else:
        a, b = r[..., :h], r[..., h:]
        out[:, :, :n, :h] = a * cos - b * sin
        out[:, :, :n, h:] = a * sin + b * cos
    return out


def _norm_plain(case, st, x, w):
    x = _heads(case, x).float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"]) * w
    return _heads(case, _rotate(case, y, st["cos"], st["sin"])).to(DTYPES[case["dtype"]])


def _norm_back_plain(case, st, dy, x, w):
    x, dy = _heads(case, x).float(), _heads(case, dy).float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + st["eps"])
    n = x * r
    g = _rotate(case, dy, st["cos"], -st["sin"])
    # the weights' gradient sums over every row: in 64 bits, three million terms of both signs
    dw = (g * n).sum((0, 1, 2), dtype=torch.float64).float()
    gw = g * w
    dx = r * (gw - n * (gw * n).mean(-1, keepdim=True))
    return _heads(case, dx).to(DTYPES[case["dtype"]]), dw


def _share(case, x):
    """Keys or values [B, Hkv, Tk, d] with every shared head repeated for its queries."""
    return _heads(case, x).float().repeat_interleave(case["H"] // case["Hkv"], 1)


def _probabilities(case, st):
    k = _share(case, st["k"])
    s = torch.matmul(_heads(case, st["q"]).float(), k.transpose(2, 3)) * (1.0 / math.sqrt(case["d"]))
    far = torch.arange(case["Tk"], device=s.device)[None, None, None, :] >= st["len"].view(-1, 1, 1, 1)
    s = s.masked_fill_(far, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    return p.div_(total), (m + total.log()).squeeze(-1)


def _cross_plain(case, st):
    p, lse = _probabilities(case, st)
    o = torch.matmul(p, _share(case, st["v"]))
    return _heads(case, o).to(DTYPES[case["dtype"]]), lse


def _cross_back_plain(case, st):
    dt = DTYPES[case["dtype"]]
    p, _ = _probabilities(case, st)
    q, do = _heads(case, st["q"]).float(), _heads(case, st["dout"]).float()
    dp = torch.matmul(do, _share(case, st["v"]).transpose(2, 3))
    dv = torch.matmul(p.transpose(2, 3), do)
    ds = dp.sub_((p * dp).sum(-1, keepdim=True)).mul_(p).mul_(1.0 / math.sqrt(case["d"]))
    dq = torch.matmul(ds, _share(case, st["k"]))
    dk = torch.matmul(ds.transpose(2, 3), q)
    B, Hkv, Tk, d = case["B"], case["Hkv"], case["Tk"], case["d"]
    dk, dv = (x.view(B, Hkv, -1, Tk, d).sum(2) for x in (dk, dv))
    return tuple(_heads(case, x).to(dt) for x in (dq, dk, dv))


def run(state):
    case, st = state["case"], state
    if own:
        return _run_own(case, st)
    if case["op"] == "norm":
        return {"q": _norm_plain(case, st, st["q"], st["wq"]), "k": _norm_plain(case, st, st["k"], st["wk"])}
    if case["op"] == "norm_back":
        dq, dwq = _norm_back_plain(case, st, st["dq"], st["q"], st["wq"])
        dk, dwk = _norm_back_plain(case, st, st["dk"], st["k"], st["wk"])
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    if case["op"] == "cross":
        o, lse = _cross_plain(case, st)
        return {"out": o, "lse": lse} if case["lse"] else {"out": o}
    dq, dk, dv = _cross_back_plain(case, st)
    return {"dq": dq, "dk": dk, "dv": dv}


def _run_own(case, st):
    import sparse_mixed_precision_b200 as da2

    if "cfg" not in st:                       # the plan and the workspace that a program keeps
        dt, layout = DTYPES[case["dtype"]], case["layout"]
        if case["op"].startswith("norm"):
            st["cfg"] = da2.norm_rope_config(case["B"], case["Hq"], case["Hk"], case["T"], case["d"], dtype=dt,
                                             T_rot=case["T_rot"], eps=st["eps"], layout=layout,
                                             half=case["style"] == "halves")
            if case["op"] == "norm_back":
                st["ws"] = da2.qk_norm_rope_workspace(st["cfg"], st["q"].device)
        else:
            st["cfg"] = da2.cross_config(case["B"], case["H"], case["Tq"], case["Tk"], case["d"],
                                         Hkv=case["Hkv"], dtype=dt, layout=layout)
            st["ws"] = da2.cross_attention_workspace(st["cfg"], st["q"].device, backward=case["op"] == "cross_back")
    cfg = st["cfg"]
    if case["op"] == "norm":
        da2.qk_norm_rope(cfg, st["q"], st["k"], st["wq"], st["wk"], st["cos"], st["sin"], st["oq"], st["ok"])
        return {"q": st["oq"], "k": st["ok"]}
    if case["op"] == "norm_back":
        da2.qk_norm_rope_backward(cfg, st["dq"], st["dk"], st["q"], st["k"], st["wq"], st["wk"], st["cos"],
                                  st["sin"], st["oq"], st["ok"], st["dwq"], st["dwk"], st["ws"])
        return {"dq": st["oq"], "dk": st["ok"], "dwq": st["dwq"], "dwk": st["dwk"]}
    if case["op"] == "cross":
        da2.cross_attention(cfg, st["q"], st["k"], st["v"], st["out"], st["ws"], kv_len=st["len"], lse=st["lse"])
        return {"out": st["out"], "lse": st["lse"]} if case["lse"] else {"out": st["out"]}
    da2.cross_attention_backward(cfg, st["dout"], st["q"], st["k"], st["v"], st["out"], st["lse"], st["dq"],
                                 st["dk"], st["dv"], st["ws"], kv_len=st["len"])
    return {"dq": st["dq"], "dk": st["dk"], "dv": st["dv"]}


def work(case):
    d = case["d"]
    if case["op"].startswith("norm"):
        rows = case["B"] * case["T"] * (case["Hq"] + case["Hk"])
        table = 2 * 4 * case["T_rot"] * (d // 2)
        moved = 2 if case["op"] == "norm" else 3      # activations read and written
        flops = (9 if case["op"] == "norm" else 18) * rows * d
        return {"bytes": moved * 2 * rows * d + table + moved * 4 * d * 2, "flops": flops}
    q = 2 * case["B"] * case["H"] * case["Tq"] * d
    kv = 2 * case["Hkv"] * d * sum(_lens(case))
    whole = 2 * case["Hkv"] * d * case["Tk"] * case["B"]
    lse = 4 * case["B"] * case["H"] * case["Tq"] if case["lse"] else 0
    product = 2 * case["H"] * case["Tq"] * d * sum(_lens(case))
    if case["op"] == "cross":
        return {"bytes": 2 * q + 2 * kv + lse, "flops": 2 * product}
    return {"bytes": 4 * q + 2 * kv + 2 * whole + lse, "flops": 5 * product}


def exact(case, seed):
    """The definitions in 64 bits, one batch entry at a time."""
    st = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(case, st)
    outs = [_exact_cross(case, st, b) for b in range(case["B"])]
    return {n: torch.stack([o[n] for o in outs]) for n in outs[0]}


def _exact_norm(case, st):
    d, n = case["d"], case["T_rot"]
    # y = M_t (w * x / rms(x)) with one rotation matrix per token: complex numbers of unit length
    turn = torch.complex(st["cos"].double(), st["sin"].double())

    def to_complex(z):
        z = z.unflatten(-1, (d // 2, 2)) if case["style"] == "pairs" else z.unflatten(-1, (2, d // 2)).mT
        return torch.complex(z[..., 0].contiguous(), z[..., 1].contiguous())

    def to_real(z):
        z = torch.stack((z.real, z.imag), -1)
        return z.flatten(-2) if case["style"] == "pairs" else z.mT.flatten(-2)

    def turned(z, f):
        if n == 0:
            return z
        z = _heads(case, z)
        z = torch.cat((to_real(to_complex(z[:, :, :n]) * f), z[:, :, n:]), 2)
        return _heads(case, z)

    res = {}
    for name in ("q", "k"):
        x, w = st[name].double(), st["w" + name].double()
        rms = torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / d + st["eps"])
        if case["op"] == "norm":
            res[name] = turned(x / rms * w, turn)
        else:
            g = turned(st["d" + name].double(), turn.conj())
            res["dw" + name] = (g * x / rms).reshape(-1, d).sum(0)
            inner = (g * w * x).sum(-1, keepdim=True)
            res["d" + name] = g * w / rms - x * inner / (d * rms ** 3)
        del x
    order = ("q", "k") if case["op"] == "norm" else ("dq", "dk", "dwq", "dwk")
    return {k: res[k] for k in order}


def _exact_cross(case, st, b):
    """One batch entry, head by head over its valid keys only."""
    L, d, group = _lens(case)[b], case["d"], case["H"] // case["Hkv"]
    H, Hkv, Tq, Tk = case["H"], case["Hkv"], case["Tq"], case["Tk"]
    one = {n: (st[n][b].transpose(0, 1) if case["layout"] == "bthd" else st[n][b]) for n in ("q", "k", "v")}
    new = lambda h, t: torch.zeros((h, t, d), dtype=torch.float64, device=st["q"].device)  # noqa: E731
    back = case["op"] == "cross_back"
    if back:
        do_all = st["dout"][b].transpose(0, 1) if case["layout"] == "bthd" else st["dout"][b]
        res = {"dq": new(H, Tq), "dk": new(Hkv, Tk), "dv": new(Hkv, Tk)}
    else:
        res = {"out": new(H, Tq)}
        if case["lse"]:
            res["lse"] = torch.zeros((H, Tq), dtype=torch.float64, device=st["q"].device)
    for h in range(H):
        q, k, v = one["q"][h].double(), one["k"][h // group, :L].double(), one["v"][h // group, :L].double()
        s = (q @ k.T) / math.sqrt(d)
        z = torch.logsumexp(s, 1)
        p = torch.exp(s - z[:, None])
        if not back:
            res["out"][h] = p @ v
            if case["lse"]:
                res["lse"][h] = z
            continue
        do = do_all[h].double()
        o = p @ v
        ds = p * (do @ v.T - (do * o).sum(1, keepdim=True)) / math.sqrt(d)
        res["dq"][h] = ds @ k
        res["dk"][h // group, :L] += ds.T @ q
        res["dv"][h // group, :L] += p.T @ do
    if case["layout"] == "bthd":
        res = {n: (x if n == "lse" else x.transpose(0, 1)) for n, x in res.items()}
    return res
