"""Definitions of the operators of include/forge_ffn.h on CPU tensors: the codes of blocks of 128 in the
32-bit operations that the header names, everything else in 64 bits."""
import math

import torch

from tests.layer_ref import F64, U, grouped, spans  # noqa: F401

FP8, I8 = torch.float8_e4m3fn, torch.int8
MOST = {FP8: 448.0, I8: 127.0}
ACTS = ("silu", "gelu", "gelu_tanh", "relu")


def blocks(x):
    """x [.., D] as [.., ceil(D / 128), 128], the last block filled up with zeros."""
    x = torch.nn.functional.pad(x, (0, -x.shape[-1] % 128))
    return x.view(*x.shape[:-1], -1, 128)


def to_code(q, kind):
    return q.to(FP8) if kind is FP8 else q.round().to(I8)


def scale_of(amax, kind):
    s = torch.maximum(amax.float() / MOST[kind], torch.tensor(2.0 ** -126))
    return torch.where(torch.isfinite(amax), s, torch.nan)


def amax_of(x, dims):
    """Largest magnitude; NaN wins."""
    return torch.where(torch.isnan(x).any(dims) if isinstance(dims, int) else torch.isnan(x).flatten(*dims).any(dims[0]),
                       torch.nan, x.abs().nan_to_num(0, float("inf")).amax(dims))


def quantize(x, kind):
    """Codes and scales of x [T, D] (fp32 operations)."""
    b = blocks(x.float())
    scale = scale_of(amax_of(b, -1), kind)
    q = torch.where(torch.isnan(scale)[..., None], 0.0, b * (1.0 / scale)[..., None])
    return to_code(q, kind).flatten(-2)[..., :x.shape[-1]].contiguous(), scale


def value(q, scale, dtype=F64):
    """What codes [T, D] stand for."""
    return (blocks(q.to(dtype)) * scale.to(dtype)[..., None]).flatten(-2)[..., :q.shape[-1]].contiguous()


def quantize_weight(w):
    """Codes [E, N, K] and scales of squares."""
    e, n, k = w.shape
    b = w.float().view(e, n // 128, 128, k // 128, 128).transpose(2, 3).flatten(-2)   # [e, nb, kb, 128 * 128]
    scale = scale_of(amax_of(b, -1), FP8)
    q = torch.where(torch.isnan(scale)[..., None], 0.0, b * (1.0 / scale)[..., None]).to(FP8)
    back = q.view(torch.uint8).view(e, n // 128, k // 128, 128, 128).transpose(2, 3).reshape(e, n, k)
    return back.contiguous().view(FP8), scale


def weight_value(q, scale):
    return q.to(F64) * scale.to(F64).repeat_interleave(128, -1).repeat_interleave(128, -2)


def act(name, g):
    """The activation and its derivative."""
    if name == "silu":
        p = torch.sigmoid(g)
        return g * p, p * (1 + g * torch.sigmoid(-g))
    if name == "relu":
        return g.clamp(min=0), (g > 0).to(g.dtype)
    if name == "gelu":
        p = 0.5 * torch.special.erfc(-g * math.sqrt(0.5))   # ndtr cancels far below zero
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    z = c * (g + 0.044715 * g ** 3)
    p, q = torch.sigmoid(2 * z), torch.sigmoid(-2 * z)
    return g * p, p + g * p * q * 2 * c * (1 + 3 * 0.044715 * g * g)


def act_error(name, g):
    """How far act and act' computed in fp32 may be off.  The logistic function's exponent is rounded three times (and
    for gelu_tanh comes of five more operations), which exp turns into |exponent| u each, relative; exp2, the
    sum, the reciprocal and the products are off by at most two steps each.  1 - p is off by what p is."""
    a, d = act(name, g)
    if name == "relu":
        return torch.zeros_like(g), torch.zeros_like(g)
    if name == "silu":
        p, x, lead = torch.sigmoid(g), g.abs(), g.abs()
    elif name == "gelu":
        # erfc's argument is rounded twice: erfc(x) of a positive x falls by at most 2 (x + 1) of itself for a unit of x;
        # erfc itself is good to 4 steps, exp2's argument to 3 roundings
        p, x, lead = 0.5 * torch.special.erfc(-g * math.sqrt(0.5)), 4 * g * g + 4 * g.abs(), g.abs() * torch.exp(-g * g / 2)
        return (x + 24) * U * a.abs() + 2.0 ** -126 * g.abs(), (x + 24) * U * (p + lead) + 2.0 ** -126 * (1 + g.abs())
    else:
        b = g.clamp(-64, 64)
        c = 2 * math.sqrt(2 / math.pi)
        x = (c * b * (1 + 0.044715 * b * b)).abs() * 4
        p = torch.sigmoid(c * b * (1 + 0.044715 * b * b))
        lead = g.abs() * c * (1 + 0.134145 * b * b)
    ep = (2 * x + 24) * U
    return ep * a.abs() + 2.0 ** -126 * g.abs(), ep * p * (1 + 2 * lead) + 2.0 ** -126 * (1 + lead)


def gated_grads(name, dh, g, u):
    """d(gate), d(up), H and how far each may be off in fp32."""
    a, s = act(name, g)
    ea, es = act_error(name, g)
    want = dh * u * s, dh * a, a * u
    off = ((dh * u).abs() * es + 4 * U * want[0].abs(), dh.abs() * ea + 2 * U * want[1].abs(),
           u.abs() * ea + 2 * U * want[2].abs())
    return want, off
