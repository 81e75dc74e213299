"""Binding of include/forge_ffn.h: the gated feed-forward block's products and their backward pass,
activation checkpoints in 8 bits, and the product of fp8 codes with a scale for each block of 128.

As in the package's other calls, this is argument marshalling only: outputs are the caller's
tensors, work is enqueued on the current stream (or `stream`), and every call raises if the
library is not built.
"""
from __future__ import annotations

import torch

from . import FP8_B128, I8_B128, Tensor, _check, _lib, _ref
from .layer import _byref, _device, _groups, _here, _mat, _stream, _vec

ACT = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}
_CODES = {torch.float8_e4m3fn: FP8_B128, torch.int8: I8_B128}


def _act(act) -> int:
    if act not in ACT:
        raise ValueError(f"act must be one of {', '.join(map(repr, ACT))} (got {act!r})")
    return ACT[act]


def _blocks(n: int) -> int:
    return -(-n // 128)


def _codes(t, what: str, dev: int, scale, scales=None):
    """A descriptor of 8-bit codes as rows of the last dimension, with `scales` float32 scales (default: one
    for each 128 columns of a row)."""
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} must be float8_e4m3fn or int8 (got {t.dtype})")
    if t.get_device() != dev:
        _here(t, what, dev)
    if not t.dim() or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if scale is None:
        raise ValueError(f"{what} needs its scales")
    cols = t.shape[-1]
    rows = t.numel() // cols if cols else 0
    return Tensor(t.data_ptr(), code, rows, cols, cols,
                  _vec(scale, f"the scale of {what}", rows * _blocks(cols) if scales is None else scales, dev))


def _kept(t, dev: int, scale, cols: int):
    """Gate and up [rows, 2 cols]."""
    if t.dtype not in _CODES:
        if scale is not None:
            raise ValueError(f"gate_up: a {t.dtype} tensor takes no scale")
        return _mat(t, "gate_up", dev)
    return _codes(t, "gate_up", dev, scale, t.numel() // max(1, 2 * cols) * 2 * _blocks(cols))


def block_quantize(x, q, scale, *, stream=None) -> None:
    """q (float8_e4m3fn or int8) and scale (float32, one for each 128 columns of a row) of x (float32 or
    bfloat16) over its last dimension (forge_block_quantize)."""
    dev = _device(x, "x")
    _check(_lib().forge_block_quantize(_byref(_mat(x, "x", dev)), _byref(_codes(q, "q", dev, scale)), _stream(stream, dev)))


def block_dequantize(q, scale, y, *, stream=None) -> None:
    """y (float32 or bfloat16) = what the codes stand for (forge_block_dequantize)."""
    dev = _device(q, "q")
    _check(_lib().forge_block_dequantize(_byref(_codes(q, "q", dev, scale)), _byref(_mat(y, "y", dev)), _stream(stream, dev)))


def _weights(W, what):
    if W.dim() not in (2, 3):
        raise ValueError(f"{what} must be [N, K] or [experts, N, K] (got {tuple(W.shape)})")
    return W.shape[0] if W.dim() == 3 else 1, W.shape[-2], W.shape[-1]


def block_quantize_weight(W, q, scale, *, qt=None, scale_t=None, stream=None) -> None:
    """q (float8_e4m3fn) and scale [..., N / 128, K / 128] of the weights W [N, K] or [experts, N, K], float32 or
    bfloat16, in squares of 128; qt [..., K, N] and scale_t: the same, transposed
    (forge_block_quantize_weight)."""
    dev = _device(W, "W")
    e, n, k = _weights(W, "W")
    squares = e * _blocks(n) * _blocks(k)
    if (qt is None) != (scale_t is None):
        raise ValueError("qt and scale_t go together: both or neither")
    if qt is not None and _weights(qt, "qt") != (e, k, n):
        raise ValueError(f"qt must hold the transposed weights of W {tuple(W.shape)} (got {tuple(qt.shape)})")
    _check(_lib().forge_block_quantize_weight(
        _byref(_mat(W, "W", dev)), e, _byref(_codes(q, "q", dev, scale, squares)),
        None if qt is None else _byref(_codes(qt, "qt", dev, scale_t, squares)), _stream(stream, dev)))


def grouped_block_gemm(X, x_scale, W, w_scale, ends, Y, *, stream=None) -> None:
    """Y[t] = X[t] W[e]^T for the rows t of group e (forge_grouped_block_gemm).  X [T, K] float8_e4m3fn with x_scale
    [T, K / 128], W [E, N, K] with w_scale [E, N / 128, K / 128], ends as grouped_gemm's; Y [T, N] bfloat16.
    The transposed weights of block_quantize_weight give the input gradient."""
    dev = _device(X, "X")
    at, n = _groups(ends, dev, W)
    _check(_lib().forge_grouped_block_gemm(
        _byref(_codes(X, "X", dev, x_scale)),
        _byref(_codes(W, "W", dev, w_scale, n * _blocks(W.shape[1]) * _blocks(W.shape[2]))), at, n,
        _byref(_mat(Y, "Y", dev)), _stream(stream, dev)))


def grouped_gated(X, W, ends, H, *, gate_up=None, gate_up_scale=None, act="silu", stream=None) -> None:
    """H[t] = act(X[t] Wg[e]^T) * (X[t] Wu[e]^T) for the rows t of group e (forge_grouped_gated).  X [T, K], W
    [E, 2 N, K] (gate rows, then up rows) and H [T, N] bfloat16.  gate_up [T, 2 N]: both products kept for
    the backward pass, bfloat16, or float8_e4m3fn or int8 with gate_up_scale [T, 2, N / 128].  act: silu,
    gelu, gelu_tanh or relu."""
    dev = _device(X, "X")
    at, n = _groups(ends, dev, W)
    if gate_up is None and gate_up_scale is not None:
        raise ValueError("gate_up_scale without gate_up")
    H_ = _mat(H, "H", dev)
    _check(_lib().forge_grouped_gated(
        _byref(_mat(X, "X", dev)), _byref(_mat(W, "W", dev)), at, n, _act(act), _byref(H_),
        None if gate_up is None else _byref(_kept(gate_up, dev, gate_up_scale, H_.cols)), _stream(stream, dev)))


def gated_backward(dH, gate_up, dgate_up, *, H=None, gate_up_scale=None, act="silu", stream=None) -> None:
    """dgate_up [T, 2 N] = (dH u act'(g), dH act(g)) and, where it is given, H = act(g) u, from dH [T, N] and
    gate_up [T, 2 N] (forge_gated_backward): float32 or bfloat16, or gate_up in codes with gate_up_scale
    [T, 2, ceil(N / 128)]."""
    dev = _device(dH, "dH")
    d = _mat(dH, "dH", dev)
    _check(_lib().forge_gated_backward(
        _byref(d), _byref(_kept(gate_up, dev, gate_up_scale, d.cols)), _act(act), _byref(_mat(dgate_up, "dgate_up", dev)),
        _ref(_mat(H, "H", dev)), _stream(stream, dev)))


def grouped_gated_dgrad(dY, W, ends, gate_up, dgate_up, *, H=None, gate_up_scale=None, act="silu", stream=None) -> None:
    """gated_backward with dH[t] = dY[t] W[e] for the rows t of group e, which is not stored
    (forge_grouped_gated_dgrad): dY [T, K], W [E, K, N] the down projection, bfloat16."""
    dev = _device(dY, "dY")
    at, n = _groups(ends, dev, W)
    _check(_lib().forge_grouped_gated_dgrad(
        _byref(_mat(dY, "dY", dev)), _byref(_mat(W, "W", dev)), at, n,
        _byref(_kept(gate_up, dev, gate_up_scale, W.shape[-1])), _act(act), _byref(_mat(dgate_up, "dgate_up", dev)),
        _ref(_mat(H, "H", dev)), _stream(stream, dev)))


# the C ABI names
forge_block_quantize = block_quantize
forge_block_dequantize = block_dequantize
forge_block_quantize_weight = block_quantize_weight
forge_grouped_block_gemm = grouped_block_gemm
forge_grouped_gated = grouped_gated
forge_gated_backward = gated_backward
forge_grouped_gated_dgrad = grouped_gated_dgrad
