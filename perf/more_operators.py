"""Measured cases of the operators of a gated feed-forward block: its forward products with the
activation (for a batch, for single tokens, over experts), its backward pass, activation checkpoints
in 8 bits and the backward passes that read them, and the fp8 matrix product with a scale for each
block of 128.

`run` computes them in plain torch operations where `own` is false and through the package's entry
points where it is true; `exact` gives the same results from the definitions in 64 bits.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

BLOCK = 128            # columns of a block of 8-bit activations; rows and columns of a block of weights
FP8_MAX = 448.0
SCALE_MIN = 2.0 ** -126
NORM_EPS = 1e-5
FP8 = torch.float8_e4m3fn


def listed():
    return [
        # a decoded token through a dense block: a pass over both projections
        {"name": "gated one token", "op": "gated", "act": "silu", "experts": 1, "tokens": 1, "n": 14336, "k": 4096,
         "saved": "none"},
        # a few decoded tokens over many small experts
        {"name": "gated experts decode", "op": "gated", "act": "silu", "experts": 64, "tokens": 96, "n": 1408,
         "k": 2048, "saved": "none"},
        # a dense block's training forward, gate and up kept in 8 bits
        {"name": "gated forward", "op": "gated", "act": "silu", "experts": 1, "tokens": 8192, "n": 14336, "k": 4096,
         "saved": "fp8"},
        # experts of an odd multiple of 128, gate and up kept whole
        {"name": "gated experts forward", "op": "gated", "act": "gelu_tanh", "experts": 32, "tokens": 16384, "n": 1408,
         "k": 2048, "saved": "bf16"},
        # the dense block's backward up to its first products, from the 8-bit checkpoint
        {"name": "gated dgrad", "op": "gated_dgrad", "act": "silu", "experts": 1, "tokens": 8192, "n": 14336, "k": 4096,
         "saved": "int8"},
        # the same over experts, from whole activations
        {"name": "gated experts dgrad", "op": "gated_dgrad", "act": "gelu_tanh", "experts": 32, "tokens": 16384,
         "n": 1408, "k": 2048, "saved": "bf16"},
        # the activation's backward alone, where the gradient of its output comes from elsewhere
        {"name": "gated backward", "op": "gated_backward", "act": "silu", "tokens": 4099, "n": 17408, "saved": "fp8"},
        # a layer's input kept in 8 bits and read back
        {"name": "checkpoint", "op": "checkpoint", "type": "int8", "tokens": 16384, "width": 5120},
        # the norm's backward from its 8-bit input
        {"name": "norm backward 8-bit", "op": "norm_backward", "type": "int8", "tokens": 8192, "width": 4096},
        # a few decoded tokens through a quantised down projection: a long contraction, few columns
        {"name": "block product decode", "op": "block", "experts": 1, "tokens": 8, "n": 4096, "k": 14336},
        # a batch over few large quantised experts
        {"name": "block product", "op": "block", "experts": 8, "tokens": 16384, "n": 14336, "k": 4096},
        # weights quantised after their step, with the transposed copy that the input gradient takes
        {"name": "block weights", "op": "block_weight", "experts": 8, "n": 14336, "k": 4096},
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_dgrad", "gated_backward", "checkpoint", "norm_backward", "block", "block",
                     "block_weight"])
    act = rng.choice(["silu", "gelu_tanh", "gelu", "relu"])
    if op == "gated_backward":
        return {"op": op, "act": act, "tokens": _log_int(rng, 1, 4000), "n": _log_int(rng, 1, 17408),
                "saved": rng.choice(["bf16", "fp8", "int8"])}
    if op in ("checkpoint", "norm_backward"):
        return {"op": op, "type": rng.choice(["fp8", "int8"]), "tokens": _log_int(rng, 1, 8192),
                "width": _log_int(rng, 128, 8192)}
    case = {"op": op, "experts": _log_int(rng, 1, 128), "n": 128 * _log_int(rng, 1, 112), "k": 128 * _log_int(rng, 1, 64)}
    while case["experts"] * case["n"] * case["k"] > 1 << 28:
        case["experts"] = (case["experts"] + 1) // 2
        case["n"] = 128 * max(1, case["n"] // 256)
    if op == "block_weight":
        return case
    case["tokens"] = _log_int(rng, 1, 32768)
    if op != "block":
        case["act"] = act
        case["saved"] = rng.choice(["bf16", "fp8", "int8"] + (["none"] if op == "gated" else []))
        if op == "gated" and case["saved"] == "int8":
            case["saved"] = "none"        # codes that are whole numbers are not compared as values
    while case["tokens"] * case["n"] * case["k"] > 1 << 38:
        case["tokens"] //= 2
    return case


def _expert_rows(case, seed):
    """Tokens of each expert: uneven, as routers give them, with some experts left empty."""
    rng = random.Random(seed)
    share = [rng.expovariate(1.0) ** 1.2 + 1e-3 for _ in range(case["experts"])]
    total, rows, left = sum(share), [], case["tokens"]
    for s in share:
        r = min(left, int(case["tokens"] * s / total))
        rows.append(r)
        left -= r
    rows[rng.randrange(len(rows))] += left
    return rows


def _blocks(x):
    """x in blocks of 128 of its last dimension, the last one filled up with zeros."""
    d = x.shape[-1]
    pad = -d % BLOCK
    x = torch.nn.functional.pad(x, (0, pad)) if pad else x
    return x.view(*x.shape[:-1], -1, BLOCK)


def _quantised(x, kind):
    """Codes and scales of float32 x in blocks of 128 columns."""
    b = _blocks(x)
    most = FP8_MAX if kind == "fp8" else 127.0
    scale = (b.abs().amax(-1) / most).clamp(min=SCALE_MIN)
    q = (b * (1.0 / scale)[..., None]).clamp(-most, most)
    q = q.to(FP8) if kind == "fp8" else q.round().to(torch.int8)
    return q.view(*x.shape[:-1], -1)[..., :x.shape[-1]].contiguous(), scale


def _value(q, scale, dtype=torch.float32):
    """What codes of blocks of 128 columns stand for."""
    return (_blocks(q.to(dtype)) * scale.to(dtype)[..., None]).flatten(-2)[..., :q.shape[-1]]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(*shape, device=dev, generator=gen).mul_(std).to(dtype)

    def loud(t, d, std=1.0):    # activations with a few loud channels
        c = 1.0 + 30.0 * (torch.rand(d, device=dev, generator=gen) < 0.002)
        return (torch.randn(t, d, device=dev, generator=gen).mul_(c * std)).bfloat16()

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, device=dev, dtype=dtype)

    def kept(t, n, how):        # gate and up as the forward pass has left them, and their scales
        x = torch.cat([loud(t, n, 1.5), loud(t, n)], 1)
        if how == "bf16":
            return x, None
        q, scale = _quantised(x.float().view(2 * t, n), how)     # blocks begin anew at up
        return q.view(t, 2 * n), scale.view(t, -1)

    op, s = case["op"], {"case": case}
    t, n, k = case.get("tokens"), case.get("n"), case.get("k")
    if op == "checkpoint":
        s["x"] = loud(t, case["width"])
        s["q"] = empty(t, case["width"], dtype=FP8 if case["type"] == "fp8" else torch.int8)
        s["scale"], s["y"] = empty(t, -(-case["width"] // BLOCK), dtype=torch.float32), empty(t, case["width"])
        return s
    if op == "norm_backward":
        d = case["width"]
        s["gain"] = 1.0 + normal(d, std=0.1, dtype=torch.float32)
        h = loud(t, d).float()
        s["rstd"] = torch.rsqrt(h.square().mean(1) + NORM_EPS)
        s["h"], s["h_scale"] = _quantised(h, case["type"])
        s["dy"], s["dh"] = normal(t, d, std=1e-2), normal(t, d, std=1e-2)
        s["dx"], s["dgain"] = empty(t, d), empty(d, dtype=torch.float32)
        if own:
            import optimizer_step_weight_amd as forge
            s["workspace"] = forge.rmsnorm_backward_workspace(t, d)
        return s
    if op == "gated_backward":
        s["gu"], s["gu_scale"] = kept(t, n, case["saved"])
        s["dH"], s["dgu"], s["H"] = normal(t, n, std=1e-2), empty(t, 2 * n), empty(t, n)
        return s
    e = case["experts"]
    if op == "block_weight":
        s["W"] = normal(e, n, k, std=k ** -0.5)
        s["q"], s["qt"] = empty(e, n, k, dtype=FP8), empty(e, k, n, dtype=FP8)
        s["scale"], s["scale_t"] = (empty(e, a // BLOCK, b // BLOCK, dtype=torch.float32) for a, b in ((n, k), (k, n)))
        return s
    s["rows"] = _expert_rows(case, seed)
    s["ends"] = torch.tensor(np.cumsum(s["rows"]), dtype=torch.int32).to(dev)
    if op == "gated":
        s["X"], s["W"], s["H"] = loud(t, k), normal(e, 2 * n, k, std=k ** -0.5), empty(t, n)
        if case["saved"] != "none":
            s["gu"] = empty(t, 2 * n, dtype=FP8 if case["saved"] == "fp8" else torch.bfloat16)
            if case["saved"] == "fp8":
                s["gu_scale"] = empty(t, 2 * n // BLOCK, dtype=torch.float32)
    elif op == "gated_dgrad":
        s["dY"], s["W"] = normal(t, k, std=1e-2), normal(e, k, n, std=n ** -0.5)
        s["gu"], s["gu_scale"] = kept(t, n, case["saved"])
        s["dgu"], s["H"] = empty(t, 2 * n), empty(t, n)
    else:
        s["X"], s["X_scale"] = _quantised(loud(t, k).float(), "fp8")
        w = normal(e, n, k, std=k ** -0.5, dtype=torch.float32).view(e, n // BLOCK, BLOCK, k // BLOCK, BLOCK)
        s["W_scale"] = (w.abs().amax((2, 4)) / FP8_MAX).contiguous()
        s["W"] = (w / s["W_scale"][:, :, None, :, None]).to(FP8).view(e, n, k)
        s["Y"] = empty(t, n)
    return s


def _act(name, g):
    """The activation and its derivative, in the type of g."""
    if name == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return g * p, p * (1.0 + g * (1.0 - p))
    if name == "relu":
        on = (g > 0).to(g.dtype)
        return g * on, on
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        th = torch.tanh(c * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * c * (1.0 + 3 * 0.044715 * g * g)
    p = 0.5 * torch.erfc(-g * math.sqrt(0.5))
    return g * p, p + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import optimizer_step_weight_amd as forge
    case = s["case"]
    op = case["op"]
    if op == "gated":
        forge.grouped_gated(s["X"], s["W"], s["ends"], s["H"], gate_up=s.get("gu"), gate_up_scale=s.get("gu_scale"),
                            act=case["act"])
        return {x: s[x] for x in ("H", "gu", "gu_scale") if x in s}
    if op == "gated_dgrad":
        forge.grouped_gated_dgrad(s["dY"], s["W"], s["ends"], s["gu"], s["dgu"], H=s["H"], gate_up_scale=s["gu_scale"],
                                  act=case["act"])
        return {"dgu": s["dgu"], "H": s["H"]}
    if op == "gated_backward":
        forge.gated_backward(s["dH"], s["gu"], s["dgu"], H=s["H"], gate_up_scale=s["gu_scale"], act=case["act"])
        return {"dgu": s["dgu"], "H": s["H"]}
    if op == "checkpoint":
        forge.block_quantize(s["x"], s["q"], s["scale"])
        forge.block_dequantize(s["q"], s["scale"], s["y"])
        return {"y": s["y"], "scale": s["scale"]}
    if op == "norm_backward":
        forge.rmsnorm_backward(s["dy"], s["h"], s["gain"], s["rstd"], s["dx"], s["dgain"], dh=s["dh"],
                               h_scale=s["h_scale"], workspace=s["workspace"])
        return {"dx": s["dx"], "dgain": s["dgain"]}
    if op == "block":
        forge.grouped_block_gemm(s["X"], s["X_scale"], s["W"], s["W_scale"], s["ends"], s["Y"])
        return s["Y"]
    forge.block_quantize_weight(s["W"], s["q"], s["scale"], qt=s["qt"], scale_t=s["scale_t"])
    return {x: s[x] for x in ("q", "scale", "qt", "scale_t")}


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    bf = torch.bfloat16
    if op == "gated":
        n, g, u = case["n"], [], []
        for x, w in zip(s["X"].float().split(s["rows"]), s["W"].float()):
            g.append(x @ w[:n].t())
            u.append(x @ w[n:].t())
        g, u = torch.cat(g), torch.cat(u)
        out = {"H": (_act(case["act"], g)[0] * u).to(bf)}
        if case["saved"] == "bf16":
            out["gu"] = torch.cat([g, u], 1).to(bf)
        elif case["saved"] == "fp8":
            out["gu"], out["gu_scale"] = _quantised(torch.cat([g, u], 1), "fp8")
        return out
    if op in ("gated_dgrad", "gated_backward"):
        n = case["n"]
        if op == "gated_backward":
            dh = s["dH"].float()
        else:
            dh = torch.cat([a @ w for a, w in zip(s["dY"].float().split(s["rows"]), s["W"].float())])
        gu = s["gu"].view(-1, n)
        gu = gu.float() if s["gu_scale"] is None else _value(gu, s["gu_scale"].view(len(gu), -1))
        g, u = gu.view(-1, 2, n).unbind(1)
        a, d = _act(case["act"], g)
        return {"dgu": torch.cat([dh * u * d, dh * a], 1).to(bf), "H": (a * u).to(bf)}
    if op == "checkpoint":
        q, scale = _quantised(s["x"].float(), case["type"])
        return {"y": _value(q, scale).to(bf), "scale": scale}
    if op == "norm_backward":
        dy, x, r = s["dy"].float(), _value(s["h"], s["h_scale"]), s["rstd"][:, None]
        a = dy * s["gain"]
        dx = r * a - x * (r * r * r * (a * x).mean(1, keepdim=True)) + s["dh"].float()
        return {"dx": dx.to(bf), "dgain": (dy * x * r).sum(0)}
    if op == "block":
        x = _value(s["X"], s["X_scale"])
        e, n, k = s["W"].shape
        w = (s["W"].float().view(e, n // BLOCK, BLOCK, k // BLOCK, BLOCK) * s["W_scale"][:, :, None, :, None]).view(e, n, k)
        return torch.cat([a @ b.t() for a, b in zip(x.split(s["rows"]), w)]).to(bf)
    e, n, k = s["W"].shape
    w = s["W"].float().view(e, n // BLOCK, BLOCK, k // BLOCK, BLOCK)
    scale = (w.abs().amax((2, 4)) / FP8_MAX).clamp(min=SCALE_MIN)
    q = (w * (1.0 / scale)[:, :, None, :, None]).clamp(-FP8_MAX, FP8_MAX).to(FP8).view(e, n, k)
    return {"q": q, "scale": scale, "qt": q.transpose(1, 2).contiguous(), "scale_t": scale.transpose(1, 2).contiguous()}


def work(case):
    op = case["op"]
    t = case.get("tokens")
    eight = {"none": 0.0, "bf16": 2.0, "fp8": 1.0 + 4.0 / BLOCK, "int8": 1.0 + 4.0 / BLOCK}
    if op == "checkpoint":      # x; codes and scales, written and read; y
        return {"bytes": t * case["width"] * (2 + 2 * eight["int8"] + 2), "flops": 5 * t * case["width"]}
    if op == "norm_backward":
        d = case["width"]
        return {"bytes": t * d * (2 + 2 + 2 + eight["int8"]) + 8 * d + 4 * t, "flops": 13 * t * d}
    n = case["n"]
    if op == "gated_backward":
        return {"bytes": t * n * (2 + 2 * eight[case["saved"]] + 4 + 2), "flops": 15 * t * n}
    e, k = case["experts"], case["k"]
    if op == "block_weight":
        return {"bytes": e * n * k * 4, "flops": 4 * e * n * k}
    live = min(e, t)            # experts that have a token
    if op == "gated":
        return {"bytes": 2 * t * k + live * n * k * 4 + 2 * t * n + 2 * t * n * eight[case["saved"]],
                "flops": 4.0 * t * n * k}
    if op == "gated_dgrad":
        return {"bytes": 2 * t * k + live * n * k * 2 + t * n * (2 * eight[case["saved"]] + 4 + 2),
                "flops": 2.0 * t * n * k}
    return {"bytes": (t * k + live * n * k) + 4 * t * k / BLOCK + 2 * t * n, "flops": 2.0 * t * n * k}


def exact(case, seed):
    """The definitions in 64 bits, on the inputs that prepare() makes."""
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    d = lambda x: s[x].to(f64)  # noqa: E731

    def amax(x, *dims):
        return x.abs().amax(dims)

    def unblocked(scale, width):
        return scale.repeat_interleave(BLOCK, -1)[..., :width]

    def act64(g):
        """The activation and its derivative, from functions that the plain form does not use."""
        if case["act"] == "silu":
            p = torch.sigmoid(g)
            return g * p, p + g * p * torch.sigmoid(-g)
        if case["act"] == "relu":
            return g.clamp(min=0.0), torch.where(g > 0, 1.0, 0.0).to(f64)
        if case["act"] == "gelu_tanh":     # (1 + tanh z) / 2 = 1 / (1 + e^-2z)
            a = 2.0 * (2.0 / math.pi) ** 0.5
            p = torch.sigmoid(a * (g + 0.044715 * g ** 3))
            return g * p, p + g * p * (1.0 - p) * a * (1.0 + 0.134145 * g ** 2)
        p = torch.special.ndtr(g)
        return g * p, p + g * (-(g ** 2) / 2).exp() / (2 * math.pi) ** 0.5

    def spans():
        ends = np.concatenate([[0], np.cumsum(s["rows"])])
        return [slice(int(a), int(b)) for a, b in zip(ends[:-1], ends[1:])]

    if op == "checkpoint":
        x, w = d("x"), case["width"]
        most = 448.0 if case["type"] == "fp8" else 127.0
        scale = torch.stack([amax(x[:, c:c + BLOCK], 1) for c in range(0, w, BLOCK)], 1) / most
        scale = scale.clamp(min=SCALE_MIN)
        at = unblocked(scale, w)
        q = (x / at).clamp(-most, most)
        # the grid's step: of e4m3 2^-3 of the power of two below, from 2^-6 on
        step = torch.ones_like(q) if case["type"] == "int8" else torch.exp2(torch.log2(q.abs().clamp(min=2.0 ** -6)).floor() - 3)
        return {"y": (q / step).round() * step * at, "scale": scale}
    if op == "norm_backward":
        width = case["width"]
        h = d("h") * unblocked(d("h_scale"), width)
        r, dy, w = d("rstd"), d("dy"), d("gain")
        unit = h * r[:, None]
        du = dy * w
        dh = r[:, None] * (du - unit * (du * unit).sum(1, keepdim=True) / width) + d("dh")
        return {"dx": dh, "dgain": (dy * unit).sum(0)}
    if op == "block_weight":
        e, n, k = s["W"].shape
        scale = torch.empty(e, n // BLOCK, k // BLOCK, dtype=f64, device="cuda")
        q = torch.empty(e, n, k, dtype=f64, device="cuda")
        for i in range(e):
            w = s["W"][i].to(f64)
            for r in range(n // BLOCK):
                rows = slice(BLOCK * r, BLOCK * (r + 1))
                scale[i, r] = (amax(w[rows].view(BLOCK, -1, BLOCK), 0, 2) / 448.0).clamp(min=SCALE_MIN)
                q[i, rows] = w[rows] / unblocked(scale[i, r], k)
        q = q.float()     # its size; the codes have 8 bits
        return {"q": q, "scale": scale, "qt": q.transpose(1, 2), "scale_t": scale.transpose(1, 2)}
    if op != "gated_backward":
        out = torch.empty(case["tokens"], case["n"], dtype=f64, device="cuda")
    n = case["n"]
    if op == "gated":
        up = torch.empty_like(out)
        for e, at in enumerate(spans()):
            w = s["W"][e].to(f64)
            out[at] = torch.matmul(s["X"][at].to(f64), w[:n].t())
            up[at] = torch.matmul(s["X"][at].to(f64), w[n:].t())
        res = {"H": act64(out)[0] * up}
        if case["saved"] == "bf16":
            res["gu"] = torch.cat([out, up], 1)
        elif case["saved"] == "fp8":
            gu = torch.cat([out, up], 1)
            scale = (amax(gu.view(case["tokens"], -1, BLOCK), 2) / 448.0).clamp(min=SCALE_MIN)
            res["gu"], res["gu_scale"] = gu / unblocked(scale, 2 * n), scale
        return res
    if op in ("gated_dgrad", "gated_backward"):
        if op == "gated_dgrad":
            for e, at in enumerate(spans()):
                out[at] = torch.matmul(s["dY"][at].to(f64), s["W"][e].to(f64))
        dh = out if op == "gated_dgrad" else d("dH")
        g, u = d("gu")[:, :n], d("gu")[:, n:]
        if s["gu_scale"] is not None:
            blocks = s["gu_scale"].shape[1] // 2
            g, u = g * unblocked(d("gu_scale")[:, :blocks], n), u * unblocked(d("gu_scale")[:, blocks:], n)
        a, slope = act64(g)
        return {"dgu": torch.cat([dh * u * slope, dh * a], 1), "H": a * u}
    x = d("X") * unblocked(d("X_scale"), case["k"])
    for e, at in enumerate(spans()):
        w = s["W"][e].to(f64) * unblocked(s["W_scale"][e].to(f64), case["k"]).repeat_interleave(BLOCK, 0)
        out[at] = torch.matmul(x[at], w.t())
    return out
