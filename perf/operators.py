"""Measured cases of the operators around a mixture-of-experts layer's training step: the RMS norm
with the residual's addition and an fp8 output (and its backward), the matrix products grouped by
expert (forward, input gradient, weight gradient, and the weight's optimizer step fused into the
weight gradient), and the optimizer's step over many tensors at once.

`run` computes them in plain torch operations where `own` is false and through the package's entry
points where it is true; `exact` gives the same results from the definitions in 64 bits.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

# 32-bit hyper-parameters, as the operators take them
LR, BETA1, BETA2, EPS, DECAY = (float(np.float32(x)) for x in (1e-3, 0.9, 0.999, 1e-8, 0.1))
NORM_EPS = 1e-5
FP8_MAX = 448.0
BLOCK = 64            # elements of a block of 8-bit states
FIRST_STEP = 100      # the optimizer's step count of a state's first pass


def listed():
    return [
        # the norm of one token before a decoded layer: latency alone
        {"name": "norm one token", "op": "norm", "tokens": 1, "width": 4096},
        # a batch's norm, to fp8 for the products after it
        {"name": "norm 16384 tokens", "op": "norm", "tokens": 16384, "width": 5120},
        # the same norm's backward in training
        {"name": "norm backward", "op": "norm_backward", "tokens": 8192, "width": 4096},
        # a few tokens over many small experts: every weight read for a token or two
        {"name": "experts decode", "op": "grouped", "type": "bf16", "experts": 64, "tokens": 96, "n": 1024, "k": 2048},
        # a batch over few large experts
        {"name": "experts forward", "op": "grouped", "type": "bf16", "experts": 8, "tokens": 16384, "n": 14336,
         "k": 4096},
        # the same in fp8 with scales for each row
        {"name": "experts forward fp8", "op": "grouped", "type": "fp8", "experts": 32, "tokens": 16384, "n": 4096,
         "k": 4096},
        # input gradient over many experts of an odd multiple of 128
        {"name": "experts dgrad", "op": "grouped_dgrad", "experts": 64, "tokens": 32768, "n": 1408, "k": 2048},
        # weight gradients kept in fp32 (accumulation over micro-batches)
        {"name": "experts wgrad", "op": "grouped_wgrad", "experts": 32, "tokens": 16384, "n": 1408, "k": 2048},
        # weight gradient and AdamW step of every expert
        {"name": "experts wgrad step", "op": "grouped_step", "experts": 8, "tokens": 8192, "n": 4096, "k": 4096},
        # a model's norm gains and biases
        {"name": "adamw gains", "op": "multi", "states": "f32", "weight": "f32", "grad": "f32", "tensors": 65,
         "smallest": 256, "largest": 5120},
        # embeddings, head and routers with 8-bit states
        {"name": "adamw 8-bit", "op": "multi", "states": "8bit", "weight": "bf16", "grad": "bf16", "tensors": 40,
         "smallest": 4096, "largest": 50_000_000},
        # fp32 weights and states, bf16 gradients, odd sizes
        {"name": "adamw fp32", "op": "multi", "states": "f32", "weight": "f32", "grad": "bf16", "tensors": 120,
         "smallest": 1000, "largest": 20_000_000},
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "grouped", "grouped_dgrad", "grouped_wgrad", "grouped_step", "multi"])
    if op in ("norm", "norm_backward"):
        return {"op": op, "tokens": _log_int(rng, 1, 20000), "width": _log_int(rng, 128, 8192)}
    if op == "multi":
        smallest = _log_int(rng, 1, 5000)
        return {"op": op, "states": rng.choice(["f32", "8bit"]), "weight": rng.choice(["f32", "bf16"]),
                "grad": rng.choice(["f32", "bf16"]), "tensors": rng.randint(1, 160), "smallest": smallest,
                "largest": _log_int(rng, smallest + 1, 20_000_000)}
    case = {"op": op, "experts": _log_int(rng, 1, 128), "tokens": _log_int(rng, 1, 32768),
            "n": 128 * _log_int(rng, 1, 64), "k": 128 * _log_int(rng, 1, 64)}
    if op == "grouped":
        case["type"] = rng.choice(["bf16", "fp8"])
    # no more than the largest listed ones: 2^38 products, 2^29 weights (2^27 where states go with them)
    most = 1 << (27 if op == "grouped_step" else 29)
    while case["experts"] * case["n"] * case["k"] > most:
        case["experts"] = (case["experts"] + 1) // 2
        case["n"] = 128 * max(1, case["n"] // 256)
    while case["tokens"] * case["n"] * case["k"] > 1 << 38:
        case["tokens"] //= 2
    return case


def _sizes(case):
    """Element counts of the optimizer's tensors: log-spaced, a third of them odd."""
    n, a, b = case["tensors"], case["smallest"], case["largest"]
    out = [int(round(a * (b / a) ** (i / max(1, n - 1)))) for i in range(n)]
    return [s | 1 if i % 3 == 0 else max(1, s & ~63) for i, s in enumerate(out)]


def _places(case):
    """Start of every tensor in the flat buffers (multiples of 64 elements), and their length."""
    at, places = 0, []
    for s in _sizes(case):
        places.append(at)
        at += -(-s // BLOCK) * BLOCK
    return places, at


def _decayed(case):
    """How many of the tensors decay: the larger half (gains and biases do not)."""
    return case["tensors"] // 2


def _expert_rows(case, seed):
    """Tokens of each expert: uneven, as routers give them, with some experts left empty."""
    rng = random.Random(seed)
    share = [rng.expovariate(1.0) ** 1.2 + 1e-3 for _ in range(case["experts"])]
    total, rows, left = sum(share), [], case["tokens"]
    for i, s in enumerate(share):
        r = min(left, int(case["tokens"] * s / total))
        rows.append(r)
        left -= r
    rows[rng.randrange(len(rows))] += left
    return rows


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(*shape, device=dev, generator=gen).mul_(std).to(dtype)

    op = case["op"]
    s = {"case": case}
    if op in ("norm", "norm_backward"):
        t, d = case["tokens"], case["width"]
        loud = 1.0 + 30.0 * (torch.rand(d, device=dev, generator=gen) < 0.002)     # a few loud channels
        s["gain"] = 1.0 + normal(d, std=0.1, dtype=torch.float32)
        if op == "norm":
            s["x"] = normal(t, d, std=0.5)
            s["residual"] = (torch.randn(t, d, device=dev, generator=gen) * loud).bfloat16()
            s["h"] = torch.empty_like(s["x"])
            s["y"] = torch.empty(t, d, device=dev, dtype=torch.float8_e4m3fn)
            s["scale"], s["rstd"] = torch.empty(t, device=dev), torch.empty(t, device=dev)
        else:
            s["h"] = (torch.randn(t, d, device=dev, generator=gen) * loud).bfloat16()
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + NORM_EPS)
            s["dy"], s["dh"] = normal(t, d, std=1e-2), normal(t, d, std=1e-2)
            s["dx"], s["dgain"] = torch.empty_like(s["h"]), torch.empty(d, device=dev)
            if own:
                import optimizer_step_weight_amd as forge
                s["workspace"] = forge.rmsnorm_backward_workspace(t, d)
        return s
    if op == "multi":
        wt = torch.float32 if case["weight"] == "f32" else torch.bfloat16
        gt = torch.float32 if case["grad"] == "f32" else torch.bfloat16
        sizes, (places, n) = _sizes(case), _places(case)
        held = torch.zeros(n, dtype=torch.bool, device=dev)                        # not the gaps between tensors
        for at, k in zip(places, sizes):
            held[at:at + k] = True
        s["step"] = FIRST_STEP
        s["W"] = normal(n, std=0.05, dtype=wt).mul_(held)
        s["g"] = normal(n, std=1e-2, dtype=gt).mul_(held)
        m = normal(n, std=1e-3, dtype=torch.float32).mul_(held)
        v = normal(n, std=1e-2, dtype=torch.float32).square_().mul_(held)
        if case["states"] == "f32":
            s["m"], s["v"] = m, v
        else:
            s["m"], s["m_scale"] = _to_codes(m, True)
            s["v"], s["v_scale"] = _to_codes(v, False)
        s["k"] = places[case["tensors"] - _decayed(case)] if _decayed(case) else n  # the flat index where decay begins
        if own:
            import optimizer_step_weight_amd as forge
            cut = lambda x, by=1: [x[a // by:a // by + -(-k // by)] for a, k in zip(places, sizes)]  # noqa: E731
            eight = case["states"] == "8bit"
            first = case["tensors"] - _decayed(case)
            s["plan"] = forge.MultiStep(cut(s["W"]), cut(s["g"]), cut(s["m"]), cut(s["v"]),
                                        m_scale=cut(s["m_scale"], BLOCK) if eight else None,
                                        v_scale=cut(s["v_scale"], BLOCK) if eight else None,
                                        group=[int(i >= first) for i in range(len(sizes))], opt="adamw")
        return s
    e, t, n, k = case["experts"], case["tokens"], case["n"], case["k"]
    s["rows"] = _expert_rows(case, seed)
    s["ends"] = torch.tensor(np.cumsum(s["rows"]), dtype=torch.int32).to(dev)
    if op != "grouped" or case["type"] == "bf16":
        if op != "grouped_wgrad":
            s["W"] = normal(e, n, k, std=k ** -0.5)
        if op != "grouped_dgrad":
            s["X"] = normal(t, k)
        if op != "grouped":
            s["dY"] = normal(t, n, std=1e-2)
    else:
        for name, shape, std in (("X", (t, k), 1.0), ("W", (e, n, k), k ** -0.5)):
            x = normal(*shape, std=std, dtype=torch.float32)
            scale = x.abs().amax(-1, keepdim=True) / FP8_MAX
            s[name], s[name + "_scale"] = (x / scale).to(torch.float8_e4m3fn), scale[..., 0].contiguous()
            del x
    if op == "grouped":
        s["Y"] = torch.empty(t, n, device=dev, dtype=torch.bfloat16)
    elif op == "grouped_dgrad":
        s["dX"] = torch.empty(t, k, device=dev, dtype=torch.bfloat16)
    elif op == "grouped_wgrad":
        s["dW"] = torch.empty(e, n, k, device=dev)
    else:
        s["step"] = FIRST_STEP
        s["m"] = normal(e, n, k, std=1e-3, dtype=torch.float32)
        s["v"] = normal(e, n, k, std=1e-2, dtype=torch.float32).square_()
    return s


def _to_codes(x, signed):
    """8-bit codes and scales of blocks of 64: absmax maps to 127 (signed) or 255, and no positive
    second moment to 0."""
    x = x.view(-1, BLOCK)
    scale = x.abs().amax(1)
    levels = 127.0 if signed else 255.0
    q = torch.round(x * torch.where(scale > 0, levels / scale, 0.0)[:, None])
    q = q.clamp(-127, 127) if signed else torch.maximum(q, (x > 0).to(q.dtype)).clamp(max=255)
    return q.to(torch.int8 if signed else torch.uint8).view(-1), scale


def _of_codes(code, scale, signed):
    return (code.view(-1, BLOCK) * (scale * (1.0 / (127.0 if signed else 255.0)))[:, None]).view(-1)


def _adamw(w, g, m, v, step, decay):
    """New weight and moments, in the type that they come in."""
    m = BETA1 * m + (1.0 - BETA1) * g
    v = BETA2 * v + (1.0 - BETA2) * g * g
    den = torch.sqrt(v * (1.0 / (1.0 - BETA2 ** step))) + EPS
    return w * (1.0 - LR * decay) - (LR / (1.0 - BETA1 ** step)) * (m / den), m, v


def _stated(s):
    """The optimizer's state as it is returned: 8-bit moments as the values that they stand for."""
    if "m_scale" not in s:
        return {"W": s["W"], "m": s["m"], "v": s["v"]}
    out = {"W": s["W"]}
    for name, levels in (("m", 127.0), ("v", 255.0)):
        value = torch.empty(s[name].shape, device="cuda", dtype=torch.bfloat16)
        torch.mul(s[name].view(-1, BLOCK), (s[name + "_scale"] * (1.0 / levels))[:, None], out=value.view(-1, BLOCK))
        out[name] = value
    return out


def _hyper(decay):
    return {"lr": LR, "beta1": BETA1, "beta2": BETA2, "eps": EPS, "weight_decay": decay}


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import optimizer_step_weight_amd as forge
    op = s["case"]["op"]
    if op == "norm":
        forge.rmsnorm(s["x"], s["gain"], s["y"], residual=s["residual"], h=s["h"], rstd=s["rstd"], y_scale=s["scale"],
                      eps=NORM_EPS)
        return {"h": s["h"], "y": s["y"], "scale": s["scale"], "rstd": s["rstd"]}
    if op == "norm_backward":
        forge.rmsnorm_backward(s["dy"], s["h"], s["gain"], s["rstd"], s["dx"], s["dgain"], dh=s["dh"],
                               workspace=s["workspace"])
        return {"dx": s["dx"], "dgain": s["dgain"]}
    if op == "grouped":
        forge.grouped_gemm(s["X"], s["W"], s["ends"], s["Y"], x_scale=s.get("X_scale"), w_scale=s.get("W_scale"))
        return s["Y"]
    if op == "grouped_dgrad":
        forge.grouped_dgrad(s["dY"], s["W"], s["ends"], s["dX"])
        return s["dX"]
    if op == "grouped_wgrad":
        forge.grouped_wgrad(s["X"], s["dY"], s["ends"], s["dW"])
        return s["dW"]
    if op == "grouped_step":
        forge.grouped_wgrad_step(s["X"], s["dY"], s["ends"], s["W"], s["m"], s["v"], opt="adamw", hyper=_hyper(DECAY),
                                 step=s["step"], seed=1, sr=False)
    else:
        s["plan"].step(step=s["step"], hyper=[_hyper(0.0), _hyper(DECAY)], sr=False)
    s["step"] += 1
    return _stated(s)


def _run_plain(s):
    op = s["case"]["op"]
    if op == "norm":
        h = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
        x = h.float()
        rstd = torch.rsqrt(x.square().mean(1) + NORM_EPS)
        y = x * rstd[:, None] * s["gain"]
        scale = y.abs().amax(1) * (1.0 / FP8_MAX)
        q = (y / scale[:, None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
        return {"h": h, "y": q, "scale": scale, "rstd": rstd}
    if op == "norm_backward":
        dy, x, r = s["dy"].float(), s["h"].float(), s["rstd"][:, None]
        a = dy * s["gain"]
        dx = r * a - x * (r * r * r * (a * x).mean(1, keepdim=True)) + s["dh"].float()
        return {"dx": dx.to(s["h"].dtype), "dgain": (dy * x * r).sum(0)}
    if op == "multi":
        eight = "m_scale" in s
        m, v = (_of_codes(s[x], s[x + "_scale"], x == "m") if eight else s[x] for x in ("m", "v"))
        w, g, k = s["W"].float(), s["g"].float(), s["k"]
        a, b = (_adamw(w[at], g[at], m[at], v[at], s["step"], d)
                for at, d in ((slice(0, k), 0.0), (slice(k, None), DECAY)))
        s["W"].copy_(torch.cat([a[0], b[0]]))
        m, v = torch.cat([a[1], b[1]]), torch.cat([a[2], b[2]])
        if eight:
            s["m"], s["m_scale"] = _to_codes(m, True)
            s["v"], s["v_scale"] = _to_codes(v, False)
        else:
            s["m"], s["v"] = m, v
        s["step"] += 1
        return _stated(s)
    rows = s["rows"]
    if op == "grouped":
        x, w = s["X"].float(), s["W"].float()
        if "X_scale" in s:
            x, w = x * s["X_scale"][:, None], w * s["W_scale"][..., None]
        return torch.cat([a @ b.t() for a, b in zip(x.split(rows), w)]).to(torch.bfloat16)
    if op == "grouped_dgrad":
        return torch.cat([a @ b for a, b in zip(s["dY"].float().split(rows), s["W"].float())]).to(torch.bfloat16)
    g = torch.stack([a.t() @ b for a, b in zip(s["dY"].float().split(rows), s["X"].float().split(rows))])
    if op == "grouped_wgrad":
        return g
    w, s["m"], s["v"] = _adamw(s["W"].float(), g, s["m"], s["v"], s["step"], DECAY)
    s["W"].copy_(w)
    s["step"] += 1
    return _stated(s)


def work(case):
    op = case["op"]
    if op in ("norm", "norm_backward"):
        t, d = case["tokens"], case["width"]
        if op == "norm":    # x, residual, gain; h, fp8 y, scale, rstd
            return {"bytes": t * d * (2 + 2 + 2 + 1) + 4 * d + 8 * t, "flops": 6 * t * d}
        return {"bytes": t * d * (2 + 2 + 2 + 2) + 8 * d + 4 * t, "flops": 12 * t * d}
    if op == "multi":
        n = sum(_sizes(case))
        w, g = (2 if case[x] == "bf16" else 4 for x in ("weight", "grad"))
        st = 4.0 if case["states"] == "f32" else 1.0 + 4.0 / BLOCK
        return {"bytes": n * (2 * w + g + 4 * st), "flops": 14 * n}
    e, t, n, k = case["experts"], case["tokens"], case["n"], case["k"]
    flops = 2.0 * t * n * k
    live = min(e, t)      # experts that have a token
    if op == "grouped":
        b = 1 if case["type"] == "fp8" else 2
        return {"bytes": b * (t * k + live * n * k) + 2 * t * n + (4 * (t + live * n) if b == 1 else 0), "flops": flops}
    if op == "grouped_dgrad":
        return {"bytes": 2 * (t * n + live * n * k + t * k), "flops": flops}
    if op == "grouped_wgrad":
        return {"bytes": 2 * (t * n + t * k) + 4 * e * n * k, "flops": flops}
    return {"bytes": 2 * (t * n + t * k) + e * n * k * (2 * 2 + 4 * 4), "flops": flops}


def exact(case, seed):
    """The definitions in 64 bits, on the inputs that prepare() makes."""
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64

    def adamw64(w, g, m, v, decay):
        m1 = BETA1 * m + (1.0 - BETA1) * g
        v1 = BETA2 * v + (1.0 - BETA2) * g ** 2
        mhat, vhat = m1 / (1.0 - BETA1 ** FIRST_STEP), v1 / (1.0 - BETA2 ** FIRST_STEP)
        return w - LR * (decay * w + mhat / (vhat.sqrt() + EPS)), m1, v1

    if op == "norm":
        stored = (s["x"].to(f64) + s["residual"].to(f64)).float().to(torch.bfloat16).to(f64)
        rms = (stored.pow(2).sum(1) / case["width"] + NORM_EPS).sqrt()
        y = stored / rms[:, None] * s["gain"].to(f64)
        scale = y.abs().max(1).values / FP8_MAX
        return {"h": stored, "y": y / scale[:, None], "scale": scale, "rstd": 1.0 / rms}
    if op == "norm_backward":
        dy, h, r, w = (s[x].to(f64) for x in ("dy", "h", "rstd", "gain"))
        unit = h * r[:, None]                                # y = unit * w
        du = dy * w
        dh = r[:, None] * (du - unit * (du * unit).sum(1, keepdim=True) / case["width"]) + s["dh"].to(f64)
        return {"dx": dh, "dgain": (dy * unit).sum(0)}
    if op == "multi":
        n = s["W"].numel()
        decay = torch.zeros(n, dtype=f64, device="cuda")
        decay[s["k"]:] = DECAY
        if "m_scale" not in s:
            w, m, v = adamw64(*(s[x].to(f64) for x in ("W", "g", "m", "v")), decay)
            return {"W": w, "m": m, "v": v}
        m = s["m"].to(f64) * s["m_scale"].to(f64).repeat_interleave(BLOCK) / 127.0
        v = s["v"].to(f64) * s["v_scale"].to(f64).repeat_interleave(BLOCK) / 255.0
        w, m, v = adamw64(s["W"].to(f64), s["g"].to(f64), m, v, decay)
        out = {"W": w}
        for name, x, levels in (("m", m, 127.0), ("v", v, 255.0)):
            x = x.view(-1, BLOCK)
            top = x.abs().max(1, keepdim=True).values
            code = (x * levels / top.clamp(min=1e-300)).round()
            if name == "v":
                code = torch.where((x > 0) & (code < 1), 1.0, code)
            out[name] = (code * top / levels).view(-1)
        return out
    ends = np.concatenate([[0], np.cumsum(s["rows"])])
    spans = [slice(int(a), int(b)) for a, b in zip(ends[:-1], ends[1:])]

    def value(name):
        return s[name].to(f64) * (s[name + "_scale"].to(f64)[..., None] if name + "_scale" in s else 1.0)

    if op in ("grouped", "grouped_dgrad"):
        left = value("X" if op == "grouped" else "dY")
        out = torch.empty(case["tokens"], case["n"] if op == "grouped" else case["k"], dtype=f64, device="cuda")
        w = value("W")
        for e, at in enumerate(spans):
            out[at] = torch.matmul(left[at], w[e].t() if op == "grouped" else w[e])
        return out
    g = torch.empty(case["experts"], case["n"], case["k"], dtype=f64, device="cuda")
    x, dy = value("X"), value("dY")
    for e, at in enumerate(spans):
        g[e] = torch.matmul(dy[at].t(), x[at])
    if op == "grouped_wgrad":
        return g
    w, m, v = adamw64(s["W"].to(f64), g, s["m"].to(f64), s["v"].to(f64), DECAY)
    return {"W": w, "m": m, "v": v}
