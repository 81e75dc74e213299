"""PyTorch autograd integration: layers whose backward pass updates their own weight (`FusedLinear`,
and `FusedExperts` over the experts of a mixture), and the RMS norm before them (`RMSNorm`).

FORGE explainer (gist.science), Technical Summary section 2 "Core Mechanism": the weight
gradient of a layer is consumed tile by tile by the optimizer and never stored.  In a PyTorch
model that means the layer's backward does the update: `FusedLinear.backward` calls the
library's `linear_backward_step`, which computes the input gradient dX = dY W with the weight as
it was (section 5 "Significance and Claims": the input gradient must be read before the update),
then runs the fused weight-gradient + optimizer step on W and its moments in place.  The layer
returns no weight gradient, so no optimizer object and no `.grad` buffer exist for it.

Limits the method imposes (section 5): a weight used by several consumers in one step (tied
embeddings, shared layers) cannot be updated by one of them, and non-element-wise steps such as
global gradient-norm clipping cannot see this weight's gradient.  Each forward of a layer must be
followed by exactly one backward before the next forward.

All arithmetic runs in the library's kernels; this module only marshals tensors.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import (grouped_dgrad, grouped_gemm, grouped_wgrad_step, linear_backward_step, rmsnorm, rmsnorm_backward,
               wgrad_step)

_STATES = {"adamw": "mv", "nadam": "mv", "radam": "mv", "lion": "m", "rmsprop": "v", "adagrad": "v",
           "sgd": "", "sgd_momentum": "m"}


def _packed(t: torch.Tensor) -> torch.Tensor:
    """t as the library takes it, contiguous from a 16-byte aligned address: a copy where it is not (a
    view into a larger tensor need not be)."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class _LinearStep(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x2d, anchor, layer):
        ctx.layer = layer
        ctx.save_for_backward(x2d)
        return x2d @ layer.weight.t()

    @staticmethod
    def backward(ctx, dy):
        (x2d,) = ctx.saved_tensors
        layer = ctx.layer
        dy = _packed(dy.to(layer.weight.dtype))
        layer.step_count += 1
        kw = dict(opt=layer.opt, hyper=layer.hyper, step=layer.step_count, seed=layer.seed,
                  m_scale=layer.m_scale, v_scale=layer.v_scale)
        if ctx.needs_input_grad[0]:
            dx = torch.empty_like(x2d)
            linear_backward_step(x2d, dy, layer.weight, dx, layer.m, layer.v, **kw)
        else:
            dx = None
            wgrad_step(x2d, dy, layer.weight, layer.m, layer.v, **kw)
        return dx, None, None


class FusedLinear(torch.nn.Module):
    """y = x W^T with W [out_features, in_features] bf16 (stochastic rounding on update) and the
    rule's moments on the device.  `in_features` and `out_features` must be multiples of 128.

    opt: one of adamw, nadam, radam, lion, rmsprop, adagrad, sgd, sgd_momentum.
    hyper: dict or object with the rule's hyper-parameters (defaults: lr 1e-3, betas 0.9 /
        0.999, eps 1e-8, no weight decay).
    state_dtype: "f32" or "int8" (block-64 absmax moments).
    seed: the stochastic-rounding key of this layer (give every layer its own).
    """

    def __init__(self, in_features: int, out_features: int, *, opt: str = "adamw",
                 hyper=None, state_dtype: str = "f32", seed: int = 0,
                 weight: Optional[torch.Tensor] = None, device="cuda"):
        super().__init__()
        if in_features % 128 or out_features % 128:
            raise ValueError("in_features and out_features must be multiples of 128")
        if opt not in _STATES:
            raise ValueError(f"unknown rule {opt!r}")
        self.in_features, self.out_features = in_features, out_features
        self.opt, self.seed = opt, int(seed)
        # hyper-parameters: any object or dict with lr, beta1, beta2, eps, weight_decay, wd_mode,
        # momentum, alpha, momentum_decay; missing fields take the library's defaults
        self.hyper = hyper if hyper is not None else {}
        if weight is None:
            weight = torch.randn(out_features, in_features, device=device) * (1.0 / in_features ** 0.5)
        self.register_buffer("weight", weight.to(device=device, dtype=torch.bfloat16).contiguous())
        shape = (out_features, in_features)
        nblk = out_features * in_features // 64
        st = _STATES[opt]

        def state(signed: bool, needed: bool):
            if not needed:
                return None, None
            if state_dtype == "f32":
                return torch.zeros(shape, device=device), None
            if state_dtype == "int8":
                return (torch.zeros(shape, dtype=torch.int8 if signed else torch.uint8, device=device),
                        torch.zeros(nblk, device=device))
            raise ValueError(f"unknown state dtype {state_dtype!r}")
        m, ms = state(True, "m" in st)
        v, vs = state(False, "v" in st)
        self.register_buffer("m", m)
        self.register_buffer("m_scale", ms)
        self.register_buffer("v", v)
        self.register_buffer("v_scale", vs)
        self.step_count = 0
        # a zero-size leaf that requires grad, so that backward runs (and the weight is updated)
        # even when the layer's input needs no gradient
        self._anchor = torch.nn.Parameter(torch.empty(0, device=device), requires_grad=True)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[-1] != self.in_features:
            raise ValueError(f"expected last dimension {self.in_features}, got {x.shape[-1]}")
        lead = x.shape[:-1]
        x2d = _packed(x.reshape(-1, self.in_features).to(torch.bfloat16))
        y = _LinearStep.apply(x2d, self._anchor, self)
        return y.reshape(*lead, self.out_features)

    def extra_repr(self) -> str:
        return f"in_features={self.in_features}, out_features={self.out_features}, opt={self.opt}"


class _ExpertsStep(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x2d, anchor, ends, layer):
        ctx.layer = layer
        ctx.save_for_backward(x2d, ends)
        y = torch.empty(x2d.shape[0], layer.out_features, dtype=torch.bfloat16, device=x2d.device)
        grouped_gemm(x2d, layer.weight, ends, y)
        return y

    @staticmethod
    def backward(ctx, dy):
        x2d, ends = ctx.saved_tensors
        layer = ctx.layer
        dy = _packed(dy.to(torch.bfloat16))
        layer.step_count += 1
        dx = None
        if ctx.needs_input_grad[0]:   # with the weights as they were
            dx = torch.empty_like(x2d)
            grouped_dgrad(dy, layer.weight, ends, dx)
        grouped_wgrad_step(x2d, dy, ends, layer.weight, layer.m, layer.v, opt=layer.opt, hyper=layer.hyper,
                           step=layer.step_count, seed=layer.seed, m_scale=layer.m_scale, v_scale=layer.v_scale)
        return dx, None, None, None


class FusedExperts(FusedLinear):
    """y[t] = x[t] W[e]^T for the rows t of expert e: FusedLinear over `experts` weights
    [experts, out_features, in_features], whose backward updates every expert's weight (one without
    rows takes a step with a zero gradient).  forward(x, ends): the rows of x are sorted by expert,
    ends[e] (int32, on the device) is the first row after expert e.  The other arguments, the limits
    and one backward for each forward are FusedLinear's."""

    def __init__(self, experts: int, in_features: int, out_features: int, *, opt: str = "adamw", hyper=None,
                 state_dtype: str = "f32", seed: int = 0, weight: Optional[torch.Tensor] = None, device="cuda"):
        if weight is not None:
            if tuple(weight.shape) != (experts, out_features, in_features):
                raise ValueError(f"weight must be [{experts}, {out_features}, {in_features}] (got {tuple(weight.shape)})")
            weight = weight.reshape(-1, in_features)
        if out_features % 128:
            raise ValueError("in_features and out_features must be multiples of 128")
        scale = 1.0 / in_features ** 0.5
        if weight is None:
            weight = torch.randn(experts * out_features, in_features, device=device) * scale
        super().__init__(in_features, experts * out_features, opt=opt, hyper=hyper, state_dtype=state_dtype, seed=seed,
                         weight=weight, device=device)
        self.experts, self.out_features = int(experts), out_features
        shape = (experts, out_features, in_features)
        for name in ("weight", "m", "v"):
            if getattr(self, name) is not None:
                setattr(self, name, getattr(self, name).view(shape))

    def forward(self, x: torch.Tensor, ends: torch.Tensor) -> torch.Tensor:
        if x.dim() != 2 or x.shape[1] != self.in_features:
            raise ValueError(f"x must be [rows, {self.in_features}] (got {tuple(x.shape)})")
        if ends.numel() != self.experts:
            raise ValueError(f"ends must have {self.experts} entries (got {ends.numel()})")
        return _ExpertsStep.apply(_packed(x.to(torch.bfloat16)), self._anchor, ends, self)

    def extra_repr(self) -> str:
        return f"experts={self.experts}, " + super().extra_repr()


class _RMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, gain, eps):
        h = None if residual is None else torch.empty_like(x)
        y = torch.empty_like(x)
        rstd = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
        rmsnorm(x, gain, y, residual=residual, h=h, rstd=rstd, eps=eps)
        ctx.save_for_backward(x if h is None else h, gain, rstd)
        ctx.alone = h is None
        ctx.set_materialize_grads(False)
        return y if h is None else (y, h)

    @staticmethod
    def backward(ctx, dy, dh=None):
        h, gain, rstd = ctx.saved_tensors
        if dy is None:   # only the stream was used
            return dh, dh, None, None
        grads = _RMSNormGrad.apply if torch.is_grad_enabled() else _norm_grads
        dx, dgain = grads(dy, dh, h, gain, rstd, ctx.needs_input_grad[2])
        return dx, None if ctx.alone else dx, dgain, None


def _norm_grads(dy, dh, h, gain, rstd, want_gain):
    dx = torch.empty_like(h)
    dgain = torch.empty(gain.shape, dtype=torch.float32, device=h.device) if want_gain else None
    rmsnorm_backward(_packed(dy), h, gain, rstd, dx, dgain, dh=None if dh is None else _packed(dh))
    return dx, None if dgain is None else dgain.to(gain.dtype)


class _RMSNormGrad(torch.autograd.Function):
    """The gradients under create_graph: connected to what they come from, so that differentiating them
    again is refused instead of passing the norm over."""

    @staticmethod
    def forward(ctx, *args):
        return _norm_grads(*args)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("RMSNorm can be differentiated once only: its gradients have no gradient")


class RMSNorm(torch.nn.Module):
    """y = h / sqrt(mean(h^2) + eps) * gain over the last dimension (float32 or bfloat16), with h = x.
    With a residual of the same shape h = x + residual, rounded to their dtype, and forward returns
    (y, h): h goes on as the residual stream.  gain is an ordinary parameter (float32).  It can be
    differentiated once: a second derivative raises."""

    def __init__(self, width: int, *, eps: float = 1e-6, device="cuda"):
        super().__init__()
        self.width, self.eps = int(width), float(eps)
        self.gain = torch.nn.Parameter(torch.ones(width, device=device))

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None):
        if x.shape[-1] != self.width:
            raise ValueError(f"expected last dimension {self.width}, got {x.shape[-1]}")
        if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype):
            raise ValueError("residual must have the shape and dtype of x")
        flat = lambda t: _packed(t.reshape(-1, self.width))  # noqa: E731
        out = _RMSNorm.apply(flat(x), None if residual is None else flat(residual), _packed(self.gain), self.eps)
        return out.view(x.shape) if residual is None else tuple(t.view(x.shape) for t in out)

    def extra_repr(self) -> str:
        return f"width={self.width}, eps={self.eps}"
