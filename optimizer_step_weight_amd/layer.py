"""Binding of include/forge_layer.h: the RMS norm with the residual's addition and an fp8 output, the
products grouped by expert, and the optimizer's step over many tensors in one launch.

As in the package's other calls, this is argument marshalling only: outputs are the caller's
tensors, work is enqueued on the current stream (or `stream`), and every call raises if the
library is not built.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import (BF16, F32, FP8_E4M3, I8_B64, I8DYN_B64, U8_B64, U8DYN_B64, Hyper, StepOpts, Tensor, _check, _dyn,
               _hyper, _lib, _opt, _opts, _ref, _stream, _tensor, _workspace)
from ._layer_abi import _MultiInfo, _MultiTensor

SCALE_MODE = {"row": 0, "tensor": 1}
_CODE = {torch.float32: F32, torch.bfloat16: BF16, torch.float8_e4m3fn: FP8_E4M3}


# The smallest calls (a norm of one token, a step of a model's gains) take less time on the device
# than their marshalling, so it asks a tensor for as little as it needs, and for the current device
# once a call.
_byref = ctypes.byref
_current_device = torch.cuda.current_device
_raw_stream = torch._C._cuda_getCurrentRawStream
_capturing = torch._C._cuda_isCurrentStreamCapturing


def _here(t: torch.Tensor, what: str, dev: int) -> None:
    at = t.get_device()
    if at != dev:
        if at < 0:
            raise ValueError(f"{what} must be a CUDA tensor (got a {t.device} tensor)")
        raise ValueError(f"{what} is on {t.device}, the current device is cuda:{dev}")


def _device(t: torch.Tensor, what: str) -> int:
    """The current device, where t has to be."""
    if t.get_device() < 0:   # asked first: without a GPU there is no current device
        raise ValueError(f"{what} must be a CUDA tensor (got a {t.device} tensor)")
    return _current_device()


def _mat(t: Optional[torch.Tensor], what: str, dev: int, scale: Optional[torch.Tensor] = None, scales: int = 0):
    """A descriptor of t as rows of its last dimension (1-D: one row), all leading dimensions
    flattened.  scale: a float32 tensor of `scales` elements (fp8 only)."""
    if t is None:
        return None
    code = _CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"{what}: unsupported dtype {t.dtype}")
    if t.get_device() != dev:
        _here(t, what, dev)
    shape = t.shape
    if not shape or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    cols = shape[-1]
    rows = shape[0] if len(shape) == 2 else t.numel() // cols if cols else 0
    at = None
    if scale is not None:
        if code != FP8_E4M3:
            raise ValueError(f"{what}: a {t.dtype} tensor takes no scale")
        at = _vec(scale, f"the scale of {what}", scales, dev)
    return Tensor(t.data_ptr(), code, rows, cols, cols, at)


def _vec(t: torch.Tensor, what: str, n: int, dev: int, dtype=torch.float32) -> int:
    """Address of a contiguous vector of n elements."""
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of {n} elements (got {t.dtype}, {t.numel()})")
    if t.get_device() != dev:
        _here(t, what, dev)
    return t.data_ptr()


def _stream(stream, dev: int) -> int:
    return _raw_stream(dev) if stream is None else int(stream)


def rmsnorm(x, gain, y, *, residual=None, h=None, rstd=None, y_scale=None, amax=None, eps: float = 1e-6,
            scale_mode: str = "row", stream=None) -> None:
    """h = x + residual, y = h / sqrt(mean(h^2) + eps) * gain over the last dimension
    (forge_rmsnorm).  y float32, bfloat16 or float8_e4m3fn; fp8 writes one scale per row to y_scale
    (scale_mode="row") or reads the tensor's one scale from it (scale_mode="tensor").  rstd (per
    row, float32) is what the backward pass takes; amax (one float32) is raised to max |y|."""
    if scale_mode not in SCALE_MODE:
        raise ValueError(f"scale_mode must be 'row' or 'tensor' (got {scale_mode!r})")
    dev = _device(x, "x")
    X = _mat(x, "x", dev)
    rows = X.rows
    _check(_lib().forge_rmsnorm(
        _byref(X), _ref(_mat(residual, "residual", dev)), _byref(_mat(gain, "gain", dev)), eps, _ref(_mat(h, "h", dev)),
        _byref(_mat(y, "y", dev, y_scale, rows if scale_mode == "row" else 1)), SCALE_MODE[scale_mode],
        None if rstd is None else _vec(rstd, "rstd", rows, dev),
        None if amax is None else _vec(amax, "amax", 1, dev), _stream(stream, dev)))


def rmsnorm_backward_workspace(rows: int, width: int, device="cuda", *, stream=None) -> torch.Tensor:
    """A workspace for rmsnorm_backward of [rows, width] tensors, allocated for work on `stream`
    (default: the current stream)."""
    n = _lib().forge_rmsnorm_backward_workspace_bytes(int(rows), int(width))
    if n < 0:
        raise ValueError(f"no workspace for [{rows}, {width}]")
    return _workspace(n // 4, torch.float32, device, stream)


def rmsnorm_backward(dy, h, gain, rstd, dx, dgain=None, *, dh=None, h_scale=None, workspace=None, stream=None) -> None:
    """dx (of x and of residual; dh, the gradient arriving on h itself, is added) and dgain
    (float32, overwritten) of rmsnorm (forge_rmsnorm_backward).  h may be 8-bit codes (float8_e4m3fn or int8)
    with h_scale, one for each 128 columns of a row, as block_quantize gives them.  A workspace is
    allocated, for the stream of the call, where dgain is wanted and none is given."""
    dev = _device(h, "h")
    if h_scale is None:
        H = _mat(h, "h", dev)
    else:
        from .ffn import _codes
        H = _codes(h, "h", dev, h_scale)
    rows, width = H.rows, H.cols
    if dgain is not None and workspace is None:
        workspace = rmsnorm_backward_workspace(rows, width, h.device, stream=stream)
    if workspace is not None:
        _here(workspace, "workspace", dev)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    _check(_lib().forge_rmsnorm_backward(
        _byref(_mat(dy, "dy", dev)), _ref(_mat(dh, "dh", dev)), _byref(H), _byref(_mat(gain, "gain", dev)),
        _vec(rstd, "rstd", rows, dev), _byref(_mat(dx, "dx", dev)), _ref(_mat(dgain, "dgain", dev)),
        None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream, dev)))


def _groups(ends, dev, W, what="W"):
    """(address of ends, number of groups); W [groups, N, K] where it is given."""
    n = ends.numel()
    if W is not None and (W.dim() != 3 or W.shape[0] != n):
        raise ValueError(f"{what} must be [experts, N, K] with one expert for each of the {n} ends "
                         f"(got {tuple(W.shape)})")
    return _vec(ends, "ends", n, dev, torch.int32), n


def grouped_gemm(X, W, ends, Y, *, x_scale=None, w_scale=None, stream=None) -> None:
    """Y[t] = X[t] W[e]^T for the rows t of group e (forge_grouped_gemm).  X [T, K] sorted by expert,
    W [E, N, K], ends [E] int32 on the device: the first row after each group.  bfloat16, or
    float8_e4m3fn X and W with x_scale [T] and w_scale [E, N]; Y [T, N] bfloat16."""
    dev = _device(X, "X")
    at, n = _groups(ends, dev, W)
    _check(_lib().forge_grouped_gemm(_byref(_mat(X, "X", dev, x_scale, X.numel() // max(1, X.shape[-1]) if X.dim() else 0)),
                                     _byref(_mat(W, "W", dev, w_scale, n * W.shape[1])), at, n,
                                     _byref(_mat(Y, "Y", dev)), _stream(stream, dev)))


def grouped_dgrad(dY, W, ends, dX, *, stream=None) -> None:
    """dX[t] = dY[t] W[e] for the rows t of group e (forge_grouped_dgrad)."""
    dev = _device(dY, "dY")
    at, n = _groups(ends, dev, W)
    _check(_lib().forge_grouped_dgrad(_byref(_mat(dY, "dY", dev)), _byref(_mat(W, "W", dev)), at, n,
                                      _byref(_mat(dX, "dX", dev)), _stream(stream, dev)))


def grouped_wgrad(X, dY, ends, dW, *, stream=None) -> None:
    """dW[e] = dY_e^T X_e in float32 for every group (forge_grouped_wgrad)."""
    dev = _device(X, "X")
    at, n = _groups(ends, dev, dW, "dW")
    _check(_lib().forge_grouped_wgrad(_byref(_mat(X, "X", dev)), _byref(_mat(dY, "dY", dev)), at, n,
                                      _byref(_mat(dW, "dW", dev)), _stream(stream, dev)))


def grouped_wgrad_step(X, dY, ends, W, m=None, v=None, *, opt="adamw", hyper=None, step: int, seed: int,
                       m_scale=None, v_scale=None, w_preround_out=None, sr=True, state_map="linear",
                       stream=None) -> None:
    """The fused step of every expert's weight: W [E, N, K], m, v updated in place from
    dW[e] = dY_e^T X_e (forge_grouped_wgrad_step; arguments as wgrad_step)."""
    dev = _device(X, "X")
    at, n = _groups(ends, dev, W)
    dyn = _dyn(state_map)
    flat = lambda t: None if t is None else t.view(-1, t.shape[-1])  # noqa: E731
    _check(_lib().forge_grouped_wgrad_step(
        _byref(_mat(X, "X", dev)), _byref(_mat(dY, "dY", dev)), at, n, _byref(_mat(W, "W", dev)),
        _ref(_tensor(flat(m), m_scale, dyn)), _ref(_tensor(flat(v), v_scale, dyn)), _byref(_hyper(hyper)), _opt(opt),
        int(step), int(seed) & 0xFFFFFFFFFFFFFFFF, _ref(_opts(w_preround_out, sr, W)), _stream(stream, dev)))


_NO_SR = _byref(StepOpts(None, 0))


class MultiStep:
    """One optimizer step over many tensors in one launch (forge_multi_pack, forge_multi_step).

    W, g: lists of contiguous float32 or bfloat16 tensors of any size (16-byte aligned).  m, v:
    their moments, all float32, or all 8-bit (int8 m, uint8 v) with m_scale / v_scale lists of
    ceil(n / 64) float32 block scales in the linear or dynamic map; None for a moment the rule does
    not keep.  group: which of step()'s hyper-parameter sets (at most 8) each tensor takes
    (default: all the first).  seed: stochastic-rounding key of each tensor (default: its index).

    The plan holds its tensors and their addresses: gradients are to be written into the same
    tensors before every step (or set_grads() called with others).  set_grads() and dropping the plan
    leave steps that are still queued on any stream as they are; that stream has to live as long as
    the plan.  A graph that captured a step goes on with the tensors of that time: it needs the plan,
    and is to be captured anew where it shall take other gradients.
    """

    def __init__(self, W: Sequence, g: Sequence, m: Optional[Sequence] = None, v: Optional[Sequence] = None, *,
                 m_scale: Optional[Sequence] = None, v_scale: Optional[Sequence] = None,
                 group: Optional[Sequence[int]] = None, seed: Optional[Sequence[int]] = None, opt="adamw",
                 state_map: str = "linear"):
        self.opt, self._dyn = _opt(opt), _dyn(state_map)
        n = len(W)
        lists = {"W": list(W)}
        for name, x in (("g", g), ("m", m), ("v", v), ("m_scale", m_scale), ("v_scale", v_scale)):
            if x is not None and len(x) != n:
                raise ValueError(f"{name} has {len(x)} tensors, W has {n}")
            lists[name] = None if x is None else list(x)
        self.group = [0] * n if group is None else [int(x) for x in group]
        self.seed = list(range(n)) if seed is None else [int(x) & 0xFFFFFFFFFFFFFFFF for x in seed]
        if len(self.group) != n or len(self.seed) != n:
            raise ValueError("group and seed take one entry for each tensor")
        self._hypers, self._given = (Hyper * 8)(), None
        self._captured = []
        self._pack(lists)

    def set_grads(self, g: Sequence) -> None:
        """Takes other gradient tensors (the table is packed and copied anew).  Where they are refused,
        the plan keeps those that it had."""
        if len(g) != len(self._lists["W"]):
            raise ValueError(f"g has {len(g)} tensors, W has {len(self._lists['W'])}")
        self._pack(dict(self._lists, g=list(g)))

    def _pack(self, L: dict) -> None:
        """Checks and packs the tensors; the plan takes them all at once, at the end."""
        n = len(L["W"])
        if L["g"] is None:
            raise ValueError("g is None")
        codes = {}
        for name, eight, dyn8, lin8 in (("m", torch.int8, I8DYN_B64, I8_B64), ("v", torch.uint8, U8DYN_B64, U8_B64)):
            kinds = {t.dtype for t in L[name]} if L[name] else set()
            if kinds - {torch.float32, eight} or len(kinds) > 1:
                raise TypeError(f"{name}: all float32 or all {eight} (got {sorted(map(str, kinds))})")
            codes[name] = F32 if not kinds or torch.float32 in kinds else (dyn8 if self._dyn else lin8)
            if L[name + "_scale"] is not None and codes[name] == F32 and n:
                raise ValueError(f"float32 {name} takes no scales")
            if L[name + "_scale"] is None and codes[name] != F32:
                raise ValueError(f"8-bit {name} needs {name}_scale")
        entries = (_MultiTensor * n)()
        dev = _device(L["W"][0], "W[0]") if n else -1
        for i, w in enumerate(L["W"]):
            count = w.numel()
            e = entries[i]
            e.n, e.seed, e.group = count, self.seed[i], self.group[i]
            for name in ("W", "g", "m", "v"):
                if L[name] is None:
                    continue
                t = L[name][i]
                if name in ("W", "g") and t.dtype not in (torch.float32, torch.bfloat16):
                    raise TypeError(f"{name}[{i}]: unsupported dtype {t.dtype}")
                setattr(e, name, _vec(t, f"{name}[{i}]", count, dev, t.dtype) or None)
            e.w_dtype, e.g_dtype = _CODE[w.dtype], _CODE[L["g"][i].dtype]
            for name in ("m_scale", "v_scale"):
                if L[name] is not None:
                    setattr(e, name, _vec(L[name][i], f"{name}[{i}]", -(-count // 64), dev) or None)
        lib = _lib()
        size = lib.forge_multi_table_bytes(entries, n)
        host = torch.empty(max(size, 16), dtype=torch.uint8)
        info = _MultiInfo()
        _check(lib.forge_multi_pack(entries, n, self.opt, codes["m"], codes["v"], host.data_ptr(), host.numel(),
                                    ctypes.byref(info)))
        # a synchronous copy: the table is there for any stream
        table = host.to(L["W"][0].device) if n else None
        self._lists, self._info, self._table, self._device = L, info, table, dev if n else None
        self._home = _stream(None, dev) if n else None   # the allocator orders the table's reuse after this one
        self._held = set()

    def _hold(self, stream: int) -> None:
        """Keeps the table and the tensors from reuse until the steps on `stream`, which is not (known to be) the
        one that the table was allocated on, are done: for good where the stream is captured into a graph."""
        s = torch.cuda.ExternalStream(stream, device=self._device)
        with torch.cuda.stream(s):
            captured = _capturing()
        if captured:
            if not self._captured or self._captured[-1][0] is not self._table:
                self._captured.append((self._table, self._lists))
        elif stream not in self._held:   # once: the allocator remembers it
            for t in [self._table, *(t for x in self._lists.values() if x is not None for t in x)]:
                t.record_stream(s)
            self._held.add(stream)

    def step(self, *, step: int, hyper=None, grad_scale: Optional[torch.Tensor] = None, sr: bool = True,
             stream=None) -> None:
        """One step: hyper is one set of hyper-parameters, or a list with one for each group;
        grad_scale one float32 on the device that multiplies every gradient."""
        hypers = list(hyper) if isinstance(hyper, (list, tuple)) else [hyper if hyper is not None else {}]
        if len(hypers) > 8:
            raise ValueError("at most 8 groups of hyper-parameters")
        if self._given is None or self._given != hypers:   # by value: they seldom change from step to step
            taken = [_hyper(h) for h in hypers]            # all of them, or none where one is refused
            for i, h in enumerate(taken):
                self._hypers[i] = h
            # comparable by value only where nothing in them can be changed in place
            plain = all(isinstance(h, dict) and all(isinstance(x, (float, int)) for x in h.values()) for h in hypers)
            self._given = [dict(h) for h in hypers] if plain else None
        dev = self._device
        table = None
        if dev is not None:
            if dev != _current_device():
                raise ValueError(f"the tensors are on cuda:{dev}, the current device is cuda:{_current_device()}")
            table = self._table.data_ptr()
            launch = _stream(stream, dev)
            if stream is not None or launch != self._home or _capturing():
                self._hold(launch)
        _check(_lib().forge_multi_step(
            _byref(self._info), table, self._hypers, len(hypers), int(step),
            None if grad_scale is None else _vec(grad_scale, "grad_scale", 1, dev),
            None if sr else _NO_SR, None if dev is None else launch))


# the C ABI names
forge_rmsnorm = rmsnorm
forge_rmsnorm_backward = rmsnorm_backward
forge_grouped_gemm = grouped_gemm
forge_grouped_dgrad = grouped_dgrad
forge_grouped_wgrad = grouped_wgrad
forge_grouped_wgrad_step = grouped_wgrad_step
