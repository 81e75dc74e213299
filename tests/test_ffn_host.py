"""Host side of include/forge_ffn.h, no GPU needed: refusals with their statuses (fake, never-dereferenced
addresses), the binding's own checks, and the gated formulas against differences in 64 bits."""
import ctypes
import os

import pytest
import torch

from tests import ffn_ref as R


@pytest.fixture(scope="module")
def f():
    import optimizer_step_weight_amd as forge
    if not os.path.exists(forge.LIB_PATH):
        from optimizer_step_weight_amd import _build
        _build.build(verbose=False)
    forge._lib()
    return forge


FAKE, GB = 0x7F0000000000, 1 << 30
ARG, SHAPE, DTYPE, LAYOUT, ALIAS = 1, 2, 3, 4, 5
r = ctypes.byref


def t(f, slot, rows, cols, dtype=None, off=0, scale=None, ld=None):
    return f.Tensor(FAKE + slot * GB + off, f.BF16 if dtype is None else dtype, rows, cols, cols if ld is None else ld,
                    scale)


def ref(x):
    return None if x is None else r(x)


def test_codes_refusals(f):
    L, T, D, S = f._lib(), 5, 300, FAKE + 9 * GB
    q = lambda dt=f.FP8_B128, scale=S, rows=T, cols=D, **k: t(f, 1, rows, cols, dt, scale=scale, **k)  # noqa: E731
    for call in (lambda x, c: L.forge_block_quantize(ref(x), ref(c), None), lambda x, c: L.forge_block_dequantize(ref(c), ref(x), None)):
        for x, c, want in [
            (None, q(), ARG), (t(f, 0, T, D), None, ARG), (t(f, 0, T, D, f.FP8_E4M3), q(), DTYPE), (t(f, 0, T, D), q(f.FP8_E4M3), DTYPE),
            (t(f, 0, T, D), q(f.I8_B64), DTYPE), (t(f, 0, T, D), q(cols=D + 1), SHAPE), (t(f, 0, T, D), q(scale=None), ARG),
            (t(f, 0, T, D), q(scale=S + 2), LAYOUT), (t(f, 0, T, D, off=8), q(), LAYOUT), (t(f, 0, T, D, ld=D + 8), q(), LAYOUT),
            (t(f, 1, T, D), q(), ALIAS), (t(f, 0, T, 0), q(cols=0), SHAPE),
        ]:
            assert call(x, c) == want, f.last_error()
        assert call(t(f, 0, 0, D), q(rows=0, scale=None)) == 0
    assert L.forge_block_quantize(r(t(f, 0, T, D)), r(q(scale=FAKE + 1 * GB + 16)), None) == ALIAS
    assert L.forge_block_quantize(r(t(f, 0, T, D)), r(q(scale=FAKE + 16)), None) == ALIAS


def test_weight_codes_refusals(f):
    L, E, N, K = f._lib(), 2, 256, 384
    S, S2 = FAKE + 8 * GB, FAKE + 9 * GB
    W, q, qt = t(f, 0, E * N, K), t(f, 1, E * N, K, f.FP8_B128, scale=S), t(f, 2, E * K, N, f.FP8_B128, scale=S2)
    call = lambda w=W, e=E, a=q, b=qt: L.forge_block_quantize_weight(ref(w), e, ref(a), ref(b), None)  # noqa: E731
    for kw, want in [
        (dict(w=None), ARG), (dict(a=None), ARG), (dict(e=0), ARG), (dict(e=3), SHAPE), (dict(w=t(f, 0, E * N, 200)), SHAPE),
        (dict(w=t(f, 0, E * N, K, f.FP8_E4M3)), DTYPE), (dict(a=t(f, 1, E * N, K, f.I8_B128, scale=S)), DTYPE),
        (dict(b=t(f, 2, E * N, K, f.FP8_B128, scale=S2)), SHAPE), (dict(a=t(f, 1, E * N, K, f.FP8_B128)), ARG),
        (dict(b=t(f, 2, E * K, N, f.FP8_B128)), ARG), (dict(b=t(f, 1, E * K, N, f.FP8_B128, scale=S2)), ALIAS),
        (dict(b=t(f, 2, E * K, N, f.FP8_B128, scale=S)), ALIAS), (dict(a=t(f, 0, E * N, K, f.FP8_B128, scale=S)), ALIAS),
    ]:
        assert call(**kw) == want, (kw, f.last_error())


def test_block_product_refusals(f):
    L, T, N, K, E = f._lib(), 70, 256, 384, 3
    S, S2, ends = FAKE + 8 * GB, FAKE + 9 * GB, FAKE + 6 * GB
    X, W, Y = t(f, 0, T, K, f.FP8_B128, scale=S), t(f, 1, E * N, K, f.FP8_B128, scale=S2), t(f, 2, T, N)
    call = lambda x=X, w=W, at=ends, n=E, y=Y: L.forge_grouped_block_gemm(ref(x), ref(w), at, n, ref(y), None)  # noqa: E731
    for kw, want in [
        (dict(x=None), ARG), (dict(w=None), ARG), (dict(y=None), ARG), (dict(at=None), ARG), (dict(n=0), ARG), (dict(at=ends + 1), LAYOUT),
        (dict(n=2), SHAPE), (dict(x=t(f, 0, T, K, f.FP8_E4M3, scale=S)), DTYPE), (dict(w=t(f, 1, E * N, K, f.I8_B128, scale=S2)), DTYPE),
        (dict(y=t(f, 2, T, N, f.F32)), DTYPE), (dict(x=t(f, 0, T, K, f.FP8_B128)), ARG), (dict(w=t(f, 1, E * N, K, f.FP8_B128)), ARG),
        (dict(x=t(f, 0, T, 200, f.FP8_B128, scale=S), w=t(f, 1, E * N, 200, f.FP8_B128, scale=S2)), SHAPE),
        (dict(y=t(f, 0, T, N)), ALIAS), (dict(x=t(f, 0, T, K, f.FP8_B128, scale=FAKE + 2 * GB)), ALIAS), (dict(at=FAKE + 2 * GB), ALIAS),
    ]:
        assert call(**kw) == want, (kw, f.last_error())
    assert call(x=t(f, 0, 0, K, f.FP8_B128), y=t(f, 2, 0, N)) == 0


def test_gated_refusals(f):
    L, T, N, K, E = f._lib(), 70, 256, 384, 3
    ends, S = FAKE + 6 * GB, FAKE + 9 * GB
    X, W, H = t(f, 0, T, K), t(f, 1, E * 2 * N, K), t(f, 2, T, N)
    G = t(f, 3, T, 2 * N, f.I8_B128, scale=S)
    call = lambda x=X, w=W, at=ends, n=E, act=0, h=H, g=G: L.forge_grouped_gated(ref(x), ref(w), at, n, act, ref(h), ref(g), None)  # noqa: E731
    for kw, want in [
        (dict(x=None), ARG), (dict(w=None), ARG), (dict(h=None), ARG), (dict(at=None), ARG), (dict(n=4097), ARG), (dict(act=4), ARG),
        (dict(act=-1), ARG), (dict(w=t(f, 1, E * N, K)), SHAPE), (dict(h=t(f, 2, T, N + 64)), SHAPE), (dict(h=t(f, 2, T + 1, N)), SHAPE),
        (dict(x=t(f, 0, T, K, f.F32)), DTYPE), (dict(h=t(f, 2, T, N, f.F32)), DTYPE), (dict(g=t(f, 3, T, N)), SHAPE),
        (dict(g=t(f, 3, T, 2 * N, f.F32)), DTYPE), (dict(g=t(f, 3, T, 2 * N, f.I8_B64, scale=S)), DTYPE),
        (dict(g=t(f, 3, T, 2 * N, f.FP8_B128)), ARG), (dict(g=t(f, 2, T, 2 * N)), ALIAS), (dict(h=t(f, 0, T, N)), ALIAS),
        (dict(g=t(f, 3, T, 2 * N, f.FP8_B128, scale=FAKE + 2 * GB)), ALIAS),
        (dict(x=t(f, 0, T, 1 << 20), w=t(f, 1, E * 2048, 1 << 20), h=t(f, 2, T, 1024), g=None), SHAPE),
    ]:
        assert call(**kw) == want, (kw, f.last_error())
    assert call(x=t(f, 0, 0, K), h=t(f, 2, 0, N), g=None) == 0


def test_gated_backward_refusals(f):
    L, T, N, K, E = f._lib(), 70, 256, 384, 3
    ends, S = FAKE + 6 * GB, FAKE + 9 * GB
    G, d, H = t(f, 1, T, 2 * N, f.FP8_B128, scale=S), t(f, 2, T, 2 * N), t(f, 3, T, N)
    call = lambda x=t(f, 0, T, N), g=G, act=0, d=d, h=H: L.forge_gated_backward(ref(x), ref(g), act, ref(d), ref(h), None)  # noqa: E731
    both = [
        (dict(g=None), ARG), (dict(d=None), ARG), (dict(act=9), ARG), (dict(g=t(f, 1, T, N)), SHAPE), (dict(d=t(f, 2, T, N)), SHAPE),
        (dict(h=t(f, 3, T, N + 1)), SHAPE), (dict(g=t(f, 1, T, 2 * N, f.F32)), DTYPE), (dict(d=t(f, 2, T, 2 * N, f.F32)), DTYPE),
        (dict(h=t(f, 3, T, N, f.F32)), DTYPE), (dict(g=t(f, 1, T, 2 * N, f.I8_B128)), ARG), (dict(d=t(f, 1, T, 2 * N)), ALIAS),
        (dict(h=t(f, 2, T, N)), ALIAS), (dict(g=t(f, 1, T, 2 * N, f.I8_B128, scale=FAKE + 2 * GB)), ALIAS),
        (dict(g=t(f, 2, T, 2 * N), d=t(f, 2, T, 2 * N, off=32)), ALIAS),
    ]
    for kw, want in both + [(dict(x=None), ARG), (dict(x=t(f, 0, T, N, f.I8_B128)), DTYPE), (dict(d=t(f, 0, T, 2 * N)), ALIAS)]:
        assert call(**kw) == want, (kw, f.last_error())
    z = lambda s, c, dt=None: t(f, s, 0, c, dt)  # noqa: E731
    assert call(x=z(0, N), g=z(1, 2 * N), d=z(1, 2 * N), h=z(0, N)) == 0 and call(x=z(0, N), g=z(1, 2 * N, f.I8_B128), d=z(2, 2 * N), h=None) == 0
    W = t(f, 4, E * K, N)
    call = lambda x=t(f, 0, T, K), w=W, at=ends, n=E, g=G, act=0, d=d, h=H: L.forge_grouped_gated_dgrad(  # noqa: E731
        ref(x), ref(w), at, n, ref(g), act, ref(d), ref(h), None)
    for kw, want in both + [(dict(x=None), ARG), (dict(w=None), ARG), (dict(at=None), ARG), (dict(w=t(f, 4, E * N, K)), SHAPE),
                            (dict(x=t(f, 0, T, K, f.F32)), DTYPE), (dict(w=t(f, 4, E * K, N, f.FP8_E4M3)), DTYPE),
                            (dict(h=t(f, 4, T, N)), ALIAS), (dict(d=t(f, 0, T, 2 * N)), ALIAS)]:
        assert call(**kw) == want, (kw, f.last_error())
    assert call(x=z(0, K), g=z(1, 2 * N), d=z(2, 2 * N), h=None) == 0


def test_norm_backward_of_codes_refusals(f):
    T, D, S = 5, 384, FAKE + 9 * GB
    L = f._lib()

    def call(h, dx=t(f, 5, T, D)):
        return L.forge_rmsnorm_backward(r(t(f, 0, T, D)), None, r(h), r(t(f, 3, 1, D, f.F32)), FAKE + 4 * GB, r(dx), None, None, 0, None)
    assert call(t(f, 2, T, D, f.I8_B128)) == ARG and call(t(f, 2, T, D, f.FP8_B128, scale=S + 1)) == LAYOUT
    assert call(t(f, 2, T, D, f.FP8_E4M3, scale=S)) == DTYPE and call(t(f, 2, T, D, f.I8_B64, scale=S)) == DTYPE
    assert call(t(f, 2, T, D, f.I8_B128, scale=FAKE + 5 * GB)) == ALIAS and call(t(f, 5, T, D, f.I8_B128, scale=S)) == ALIAS


def test_binding_checks_before_the_library(f):
    """CPU tensors, and arguments that go together, raise in the binding."""
    x, q, s = torch.zeros(2, 256, dtype=torch.bfloat16), torch.zeros(2, 256, dtype=torch.int8), torch.zeros(2, 2)
    w = torch.zeros(1, 256, 256, dtype=torch.bfloat16)
    ends = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: f.block_quantize(x, q, s), lambda: f.block_dequantize(q, s, x),
                 lambda: f.block_quantize_weight(w, q, s), lambda: f.grouped_gated(x, w, ends, x),
                 lambda: f.gated_backward(x, x, x), lambda: f.grouped_gated_dgrad(x, w, ends, x, x),
                 lambda: f.grouped_block_gemm(q, s, w, s, ends, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    from optimizer_step_weight_amd import ffn
    with pytest.raises(ValueError, match="silu"):
        ffn._act("swish")
    with pytest.raises(ValueError, match="scales"):
        ffn._codes(q, "q", -1, None)
    with pytest.raises(TypeError):
        ffn._codes(x, "q", -1, s)
    with pytest.raises(ValueError, match="4 elements"):
        ffn._codes(q, "q", -1, torch.zeros(5))
    with pytest.raises(ValueError, match="contiguous"):
        ffn._codes(q[:, ::2], "q", -1, s)


@pytest.mark.parametrize("act", R.ACTS)
def test_gated_formula_against_differences(act):
    g = torch.linspace(-6, 6, 401, dtype=R.F64) + 1e-3
    u, dh, h = torch.full_like(g, 0.7), torch.full_like(g, -1.3), 1e-6
    (dg, du, H), _ = R.gated_grads(act, dh, g, u)
    num = dh * u * (R.act(act, g + h)[0] - R.act(act, g - h)[0]) / (2 * h)
    assert float((dg - num).abs().max()) < 1e-8
    assert torch.equal(du, dh * R.act(act, g)[0]) and torch.equal(H, R.act(act, g)[0] * u)


def test_codes_are_within_half_a_step():
    """The rule that the GPU tests take as the reference: values come back within half a step."""
    x = torch.randn(20, 300, generator=torch.Generator().manual_seed(1)) * torch.logspace(-30, 30, 20)[:, None]
    for kind in (R.FP8, R.I8):
        q, s = R.quantize(x, kind)
        top = s.to(R.F64).repeat_interleave(128, 1)[:, :300]
        step = 2.0 ** -4 * x.to(R.F64).abs() + 2.0 ** -10 * top if kind is R.FP8 else 0.5 * top
        assert bool(((R.value(q, s) - x.to(R.F64)).abs() <= step * (1 + 1e-4)).all())


# ------------------------------------------------------------------ the layers, with stand-ins for the library
@pytest.fixture()
def A(monkeypatch):
    from optimizer_step_weight_amd import autograd

    def fine(*tensors):
        for t in tensors:
            assert t is None or (t.data_ptr() % 16 == 0 and t.is_contiguous())

    def grouped_gated(X, W, ends, H, *, gate_up=None, gate_up_scale=None, act):
        fine(X, W, H, gate_up)
        gu, _ = R.grouped(X, W, ends, True)
        n = H.shape[1]
        H.copy_(R.act(act, gu[:, :n])[0] * gu[:, n:])
        if gate_up is None:
            return
        if gate_up_scale is None:
            gate_up.copy_(gu)
        else:
            q, s = R.quantize(gu, gate_up.dtype)
            gate_up.copy_(q)
            gate_up_scale.copy_(s.view(gate_up_scale.shape))

    def grouped_gated_dgrad(dY, W, ends, gate_up, dgate_up, *, H=None, gate_up_scale=None, act):
        fine(dY, W, gate_up, dgate_up, H)
        v = gate_up.to(R.F64) if gate_up_scale is None else R.value(gate_up, gate_up_scale)
        n = H.shape[1]
        (dg, du, h), _ = R.gated_grads(act, R.grouped(dY, W, ends, False)[0], v[:, :n], v[:, n:])
        dgate_up.copy_(torch.cat([dg, du], 1))
        H.copy_(h)
    steps = []
    monkeypatch.setattr(autograd, "grouped_gated", grouped_gated)
    monkeypatch.setattr(autograd, "grouped_gated_dgrad", grouped_gated_dgrad)
    monkeypatch.setattr(autograd, "grouped_gemm", lambda X, W, ends, Y: Y.copy_(R.grouped(X, W, ends, True)[0]))
    monkeypatch.setattr(autograd, "grouped_dgrad", lambda X, W, ends, Y: Y.copy_(R.grouped(X, W, ends, False)[0]))
    monkeypatch.setattr(autograd, "grouped_wgrad_step", lambda X, dY, ends, W, *a, **k: steps.append((X.clone(), dY.clone(), W, k)))
    monkeypatch.setattr(autograd, "block_quantize", lambda x, q, s: [a.copy_(b) for a, b in zip((q, s), R.quantize(x, q.dtype))])
    monkeypatch.setattr(autograd, "block_dequantize", lambda q, s, y: y.copy_(R.value(q, s)))
    return autograd, steps


@pytest.mark.parametrize("how", [None, "int8", "fp8"])
def test_gated_layer_gradients(A, how):
    """The input's gradient and what the weights' steps are given, against autograd in 64 bits."""
    A, steps = A
    T, K, N, E = 9, 128, 256, 2
    torch.manual_seed(1)
    layer = A.FusedGatedExperts(E, K, N, act="silu", checkpoint=how, device="cpu")
    x, dy = torch.randn(T + 1, K)[1:].to(torch.bfloat16).requires_grad_(True), torch.randn(T, K).to(torch.bfloat16)
    ends = torch.tensor([4, T], dtype=torch.int32)
    layer(x, ends).backward(dy)
    assert layer.gate_up.step_count == layer.down.step_count == 1 and [k["seed"] for *_, k in steps] == [1, 0]
    x64 = x.detach().double().requires_grad_(True)
    ws = [layer.gate_up.weight.detach().double().requires_grad_(True), layer.down.weight.detach().double().requires_grad_(True)]
    out = []
    for e, (a, b) in enumerate(((0, 4), (4, T))):
        g, u = (x64[a:b] @ ws[0][e].t()).split(N, 1)
        out.append((torch.nn.functional.silu(g) * u) @ ws[1][e].t())
    torch.cat(out).backward(dy.double())
    # relative to the largest: bf16 in several places, and codes within 1 / 254 or 1 / 16 of theirs
    slack = {None: 0.02, "int8": 0.04, "fp8": 0.2}[how]
    near = lambda a, b: float((a.double() - b).abs().max()) <= slack * float(b.abs().max())  # noqa: E731
    assert near(x.grad, x64.grad)
    for (X, dY, W, _), w in zip(steps, (ws[1], ws[0])):
        dW = torch.stack([dY[a:b].double().t() @ X[a:b].double() for a, b in ((0, 4), (4, T))])
        assert near(dW, w.grad)


def test_gated_layer_without_gradients(A, monkeypatch):
    """Under no_grad the same output, nothing kept, no step; a captured training step is refused."""
    A, steps = A
    torch.manual_seed(2)
    layer = A.FusedGatedExperts(1, 128, 128, act="gelu", device="cpu")
    x = torch.randn(3, 5, 128).to(torch.bfloat16)
    y = layer(x)
    real, kept = A.grouped_gated, []
    monkeypatch.setattr(A, "grouped_gated", lambda *a, **k: (kept.append(k.get("gate_up")), real(*a, **k)))
    with torch.no_grad():
        z = layer(x)
    assert torch.equal(y, z) and z.grad_fn is None and not steps and layer.down.step_count == 0 and kept == [None]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    layer(x)                                      # a CPU tensor is on no stream
    monkeypatch.setattr(A, "_packed", lambda t: type("OnGPU", (), {"is_cuda": True, "shape": t.shape})())
    with pytest.raises(RuntimeError, match="step count"):
        layer(x)


def test_gated_layer_arguments(A):
    A, _ = A
    for kw in (dict(act="swish"), dict(checkpoint="int4"), dict(hidden=200), dict(width=100)):
        with pytest.raises(ValueError):
            A.FusedGatedExperts(**dict(dict(experts=1, width=128, hidden=128, device="cpu"), **kw))
    layer = A.FusedGatedExperts(2, 128, 128, device="cpu")
    for args in ((torch.zeros(3, 64),), (torch.zeros(3, 128),), (torch.zeros(3, 128), torch.zeros(3, dtype=torch.int32)),
                 (torch.zeros(1, 3, 128), torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            layer(*args)
    for make in (lambda: A.FusedLinear(128, 128, checkpoint="no", device="cpu"), lambda: A.RMSNorm(8, checkpoint="no", device="cpu")):
        with pytest.raises(ValueError, match="checkpoint"):
            make()
