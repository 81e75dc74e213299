"""PyTorch autograd integration: layers whose backward pass updates their own weight (`FusedLinear`,
`FusedExperts` over the experts of a mixture, and `FusedGatedExperts`, a gated feed-forward block of two
such layers), and the RMS norm before them (`RMSNorm`).

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

Layers take `checkpoint`: "int8" or "fp8" keeps what their backward pass needs of the activations in 8
bits, in blocks of 128 columns with a scale each, instead of whole.

All arithmetic runs in the library's kernels; this module only marshals tensors.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import (block_dequantize, block_quantize, grouped_dgrad, grouped_gated, grouped_gated_dgrad, grouped_gemm,
               grouped_wgrad_step, linear_backward_step, rmsnorm, rmsnorm_backward, wgrad_step)

_STATES = {"adamw": "mv", "nadam": "mv", "radam": "mv", "lion": "m", "rmsprop": "v", "adagrad": "v",
           "sgd": "", "sgd_momentum": "m"}


def _packed(t: torch.Tensor) -> torch.Tensor:
    """t as the library takes it, contiguous from a 16-byte aligned address: a copy where it is not (a
    view into a larger tensor need not be)."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


_CODES = {"int8": torch.int8, "fp8": torch.float8_e4m3fn}


def _checkpoint(how):
    """The type of the codes that activations are kept in, or None."""
    if how is not None and how not in _CODES:
        raise ValueError(f"checkpoint must be None, 'int8' or 'fp8' (got {how!r})")
    return None if how is None else _CODES[how]


def _codes_now(layer):
    """The type of a layer's codes in this call: without gradients nothing is kept.  (Asked in the module: within a
    function of autograd's gradients are off.)"""
    return layer.codes if torch.is_grad_enabled() else None


def _keep(x2d: torch.Tensor, codes):
    """x2d as it is kept for the backward pass: itself, or its codes and their scales."""
    if codes is None:
        return (x2d,)
    q = torch.empty(x2d.shape, dtype=codes, device=x2d.device)
    scale = torch.empty(x2d.shape[0], -(-x2d.shape[1] // 128), device=x2d.device)
    block_quantize(x2d, q, scale)
    return q, scale


def _kept(saved) -> torch.Tensor:
    """What _keep was given (bfloat16), as far as its codes say."""
    if len(saved) == 1:
        return saved[0]
    x2d = torch.empty(saved[0].shape, dtype=torch.bfloat16, device=saved[0].device)
    block_dequantize(*saved, x2d)
    return x2d


class _Once(torch.autograd.Function):
    """The tensor in `out`, computed by the library, connected to the tensors that it depends on under create_graph, so
    that differentiating it again is refused instead of passing the layer over."""

    @staticmethod
    def forward(ctx, out, *sources):
        return out[0]

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("this layer can be differentiated once only: its gradients have no gradient")


def _once(dx, *sources):
    return dx if dx is None or not torch.is_grad_enabled() else _Once.apply([dx], *sources)


class _LinearStep(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x2d, anchor, layer, codes):
        ctx.layer = layer
        ctx.save_for_backward(*_keep(x2d, codes))
        return x2d @ layer.weight.t()

    @staticmethod
    def backward(ctx, dy):
        x2d = _kept(ctx.saved_tensors)
        layer, arriving = ctx.layer, dy
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
        return _once(dx, arriving), None, None, None


class FusedLinear(torch.nn.Module):
    """y = x W^T with W [out_features, in_features] bf16 (stochastic rounding on update) and the
    rule's moments on the device.  `in_features` and `out_features` must be multiples of 128.

    opt: one of adamw, nadam, radam, lion, rmsprop, adagrad, sgd, sgd_momentum.
    hyper: dict or object with the rule's hyper-parameters (defaults: lr 1e-3, betas 0.9 /
        0.999, eps 1e-8, no weight decay).
    state_dtype: "f32" or "int8" (block-64 absmax moments).
    seed: the stochastic-rounding key of this layer (give every layer its own).
    checkpoint: None, "int8" or "fp8": how the input is kept for the backward pass.

    The input's gradient dY W can be differentiated once: where the arriving gradient dY depends on what it is
    differentiated by, a second derivative raises.
    """

    def __init__(self, in_features: int, out_features: int, *, opt: str = "adamw",
                 hyper=None, state_dtype: str = "f32", seed: int = 0,
                 weight: Optional[torch.Tensor] = None, checkpoint: Optional[str] = None, device="cuda"):
        super().__init__()
        self.codes = _checkpoint(checkpoint)
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
        y = _LinearStep.apply(x2d, self._anchor, self, _codes_now(self))
        return y.reshape(*lead, self.out_features)

    def extra_repr(self) -> str:
        return f"in_features={self.in_features}, out_features={self.out_features}, opt={self.opt}"


class _ExpertsStep(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x2d, anchor, ends, layer, codes):
        ctx.layer = layer
        ctx.save_for_backward(ends, *_keep(x2d, codes))
        y = torch.empty(x2d.shape[0], layer.out_features, dtype=torch.bfloat16, device=x2d.device)
        grouped_gemm(x2d, layer.weight, ends, y)
        return y

    @staticmethod
    def backward(ctx, dy):
        ends, *saved = ctx.saved_tensors
        x2d = _kept(saved)
        layer, arriving = ctx.layer, dy
        dy = _packed(dy.to(torch.bfloat16))
        dx = None
        if ctx.needs_input_grad[0]:   # with the weights as they were
            dx = torch.empty_like(x2d)
            grouped_dgrad(dy, layer.weight, ends, dx)
        _step_experts(layer, x2d, dy, ends)
        return _once(dx, arriving), None, None, None, None


def _step_experts(layer, x2d, dy, ends) -> None:
    layer.step_count += 1
    grouped_wgrad_step(x2d, dy, ends, layer.weight, layer.m, layer.v, opt=layer.opt, hyper=layer.hyper,
                       step=layer.step_count, seed=layer.seed, m_scale=layer.m_scale, v_scale=layer.v_scale)


class FusedExperts(FusedLinear):
    """y[t] = x[t] W[e]^T for the rows t of expert e: FusedLinear over `experts` weights
    [experts, out_features, in_features], whose backward updates every expert's weight (one without
    rows takes a step with a zero gradient).  forward(x, ends): the rows of x are sorted by expert,
    ends[e] (int32, on the device) is the first row after expert e.  The other arguments, the limits
    and one backward for each forward are FusedLinear's."""

    def __init__(self, experts: int, in_features: int, out_features: int, *, opt: str = "adamw", hyper=None,
                 state_dtype: str = "f32", seed: int = 0, weight: Optional[torch.Tensor] = None,
                 checkpoint: Optional[str] = None, device="cuda"):
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
                         weight=weight, checkpoint=checkpoint, device=device)
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
        return _ExpertsStep.apply(_packed(x.to(torch.bfloat16)), self._anchor, ends, self, _codes_now(self))

    def extra_repr(self) -> str:
        return f"experts={self.experts}, " + super().extra_repr()


class _GatedStep(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x2d, anchor, ends, layer):
        ctx.layer = layer
        up, down, rows = layer.gate_up, layer.down, x2d.shape[0]
        new = lambda n, dt=torch.bfloat16: torch.empty(rows, n, dtype=dt, device=x2d.device)  # noqa: E731
        hidden, y = new(layer.hidden), new(down.out_features)
        kept, scale = new(2 * layer.hidden, up.codes or torch.bfloat16), None
        if up.codes is not None:
            scale = new(2 * layer.hidden // 128, torch.float32)
        grouped_gated(x2d, up.weight, ends, hidden, gate_up=kept, gate_up_scale=scale, act=layer.act)
        grouped_gemm(hidden, down.weight, ends, y)   # `hidden` is not kept: the backward pass has it from gate and up
        # with codes an empty output: saved, it connects the gradient to x, as x itself does
        tie = None if up.codes is None else new(0)
        ctx.save_for_backward(ends, kept, scale, tie, *_keep(x2d, up.codes))
        return y, tie

    @staticmethod
    def backward(ctx, dy, _):
        ends, kept, scale, tie, *saved = ctx.saved_tensors
        layer, arriving = ctx.layer, dy
        up, down = layer.gate_up, layer.down
        dy = _packed(dy.to(torch.bfloat16))
        grad = torch.empty(kept.shape, dtype=torch.bfloat16, device=kept.device)
        hidden = torch.empty(kept.shape[0], layer.hidden, dtype=torch.bfloat16, device=kept.device)
        grouped_gated_dgrad(dy, down.weight, ends, kept, grad, H=hidden, gate_up_scale=scale, act=layer.act)
        _step_experts(down, hidden, dy, ends)
        del hidden
        dx = None
        if ctx.needs_input_grad[0]:
            dx = torch.empty(kept.shape[0], up.in_features, dtype=torch.bfloat16, device=kept.device)
            grouped_dgrad(grad, up.weight, ends, dx)
        _step_experts(up, _kept(saved), grad, ends)
        return _once(dx, arriving, tie, saved[0]), None, None, None


class _GatedServe(torch.autograd.Function):
    """The output alone.  A function of autograd's because no_grad leaves forward-mode differentiation on, which it refuses."""

    @staticmethod
    def forward(ctx, x2d, ends, layer):
        hidden = torch.empty(x2d.shape[0], layer.hidden, dtype=torch.bfloat16, device=x2d.device)
        y = torch.empty_like(x2d)
        grouped_gated(x2d, layer.gate_up.weight, ends, hidden, act=layer.act)
        grouped_gemm(hidden, layer.down.weight, ends, y)
        return y


class FusedGatedExperts(torch.nn.Module):
    """y[t] = (act(x[t] Wg[e]^T) * (x[t] Wu[e]^T)) Wd[e]^T for the rows t of expert e: a gated feed-forward
    block whose backward pass updates its weights, those of `gate_up` [experts, 2 hidden, width] (gate
    rows, then up rows) and of `down` [experts, width, hidden], both FusedExperts.  width and hidden are
    multiples of 128.  act: silu, gelu, gelu_tanh or relu.  checkpoint: None, "int8" or "fp8": how gate,
    up and the input are kept; the product of gate and up is not kept at all.  The other arguments, the limits
    and one backward for each forward are FusedLinear's; seed goes to gate_up and seed + 1 to down.  It can be differentiated
    once: a second derivative raises.

    forward(x, ends): the rows of x [rows, width] are sorted by expert, ends[e] (int32, on the device) is the
    first row after expert e.  With one expert (a dense block) ends may be left out, and x have any leading
    dimensions.  Under torch.no_grad() nothing is kept, and the call may be captured into a graph; a training step
    may not (its step count is the host's)."""

    def __init__(self, experts: int, width: int, hidden: int, *, act: str = "silu", opt: str = "adamw", hyper=None,
                 state_dtype: str = "f32", seed: int = 0, checkpoint: Optional[str] = None, device="cuda"):
        super().__init__()
        from .ffn import _act
        _act(act)
        if hidden % 128:
            raise ValueError("width and hidden must be multiples of 128")
        kw = dict(opt=opt, hyper=hyper, state_dtype=state_dtype, checkpoint=checkpoint, device=device)
        self.act, self.width, self.hidden = act, int(width), int(hidden)
        self.gate_up = FusedExperts(experts, width, 2 * hidden, seed=seed, **kw)
        self.down = FusedExperts(experts, hidden, width, seed=seed + 1, **kw)

    def forward(self, x: torch.Tensor, ends: Optional[torch.Tensor] = None) -> torch.Tensor:
        if x.shape[-1] != self.width:
            raise ValueError(f"expected last dimension {self.width}, got {x.shape[-1]}")
        lead = x.shape[:-1]
        if ends is None:
            if self.gate_up.experts != 1:
                raise ValueError(f"{self.gate_up.experts} experts need ends")
            x = x.reshape(-1, self.width)
            ends = torch.full((1,), x.shape[0], dtype=torch.int32, device=x.device)
        elif x.dim() != 2 or ends.numel() != self.gate_up.experts:
            raise ValueError(f"with ends [{self.gate_up.experts}], x must be [rows, {self.width}] "
                             f"(got {ends.numel()} ends, {tuple(x.shape)})")
        x = _packed(x.to(torch.bfloat16))
        if torch.is_grad_enabled():
            if x.is_cuda and torch.cuda.is_current_stream_capturing():
                raise RuntimeError("a captured training step would repeat its step count: capture the library's calls instead")
            y, _ = _GatedStep.apply(x, self.gate_up._anchor, ends, self)
        else:
            y = _GatedServe.apply(x, ends, self)
        return y.reshape(*lead, self.width)

    def extra_repr(self) -> str:
        return f"width={self.width}, hidden={self.hidden}, act={self.act}"


class _RMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, gain, eps, codes):
        h = None if residual is None else torch.empty_like(x)
        y = torch.empty_like(x)
        rstd = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
        rmsnorm(x, gain, y, residual=residual, h=h, rstd=rstd, eps=eps)
        if not any(ctx.needs_input_grad):
            codes = None
        # with codes an empty output: saved, it connects the gradients to x and residual, as h does where it is kept whole
        tie = None if codes is None else torch.empty(0, device=x.device)
        ctx.save_for_backward(gain, rstd, tie, *_keep(x if h is None else h, codes))
        ctx.alone = h is None
        ctx.set_materialize_grads(False)
        return (y, tie) if h is None else (y, tie, h)

    @staticmethod
    def backward(ctx, dy, _, dh=None):
        gain, rstd, tie, *h = ctx.saved_tensors
        if dy is None:   # only the stream was used
            return dh, dh, None, None, None
        grads = _RMSNormGrad.apply if torch.is_grad_enabled() else _norm_grads
        dx, dgain = grads(dy, dh, gain, rstd, tie, ctx.needs_input_grad[2], *h)
        return dx, None if ctx.alone else dx, dgain, None, None


def _norm_grads(dy, dh, gain, rstd, tie, want_gain, h, scale=None):
    dx = torch.empty(h.shape, dtype=dy.dtype, device=h.device)
    dgain = torch.empty(gain.shape, dtype=torch.float32, device=h.device) if want_gain else None
    rmsnorm_backward(_packed(dy), h, gain, rstd, dx, dgain, dh=None if dh is None else _packed(dh),
                     **({} if scale is None else {"h_scale": scale}))
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
    (y, h): h goes on as the residual stream.  gain is an ordinary parameter (float32).  checkpoint: None, "int8" or
    "fp8": how h is kept for the backward pass.  It can be differentiated once: a second derivative raises."""

    def __init__(self, width: int, *, eps: float = 1e-6, checkpoint: Optional[str] = None, device="cuda"):
        super().__init__()
        self.codes = _checkpoint(checkpoint)
        self.width, self.eps = int(width), float(eps)
        self.gain = torch.nn.Parameter(torch.ones(width, device=device))

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None):
        if x.shape[-1] != self.width:
            raise ValueError(f"expected last dimension {self.width}, got {x.shape[-1]}")
        if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype):
            raise ValueError("residual must have the shape and dtype of x")
        flat = lambda t: _packed(t.reshape(-1, self.width))  # noqa: E731
        y, _, *h = _RMSNorm.apply(flat(x), None if residual is None else flat(residual), _packed(self.gain), self.eps,
                                  _codes_now(self))
        return y.view(x.shape) if residual is None else (y.view(x.shape), h[0].view(x.shape))

    def extra_repr(self) -> str:
        return f"width={self.width}, eps={self.eps}"
