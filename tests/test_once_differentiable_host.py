"""Second derivatives of the autograd layers on the CPU, with stand-ins for the library's calls: what the library computes
has no graph, so a gradient that depends on what it is differentiated by raises, in every way that it can be kept."""
import pytest
import torch

from tests import ffn_ref as R
from tests import layer_ref as L


@pytest.fixture()
def A(monkeypatch):
    from optimizer_step_weight_amd import autograd

    def rmsnorm(x, gain, y, *, residual=None, h=None, rstd=None, eps):
        s = x.detach() if residual is None else (x.detach().float() + residual.detach().float()).to(x.dtype)
        out, r = L.norm(s.double(), gain.detach().double(), eps)
        y.data.copy_(out), rstd.data.copy_(r)
        if h is not None:
            h.data.copy_(s)

    def rmsnorm_backward(dy, h, gain, rstd, dx, dgain=None, *, dh=None, h_scale=None):
        h = h.detach().double() if h_scale is None else R.value(h, h_scale)
        gx, gg = L.norm_grads(dy.detach().double(), h, gain.detach().double(), rstd.detach().double(),
                              None if dh is None else dh.detach().double())
        dx.data.copy_(gx)
        if dgain is not None:
            dgain.data.copy_(gg)
    monkeypatch.setattr(autograd, "rmsnorm", rmsnorm)
    monkeypatch.setattr(autograd, "rmsnorm_backward", rmsnorm_backward)
    monkeypatch.setattr(autograd, "block_quantize",
                        lambda x, q, s: [a.copy_(b) for a, b in zip((q, s), R.quantize(x.detach(), q.dtype))])
    return autograd


HOW = [None, "int8", "fp8"]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("frozen", [False, True])
@pytest.mark.parametrize("linear", [False, True])
@pytest.mark.parametrize("how", HOW)
def test_norm(A, how, linear, frozen, residual):
    """Also where only the kept input ties the gradient to x: a constant gradient arrives, and the gain is frozen."""
    torch.manual_seed(1)
    norm = A.RMSNorm(200, checkpoint=how, device="cpu")
    norm.gain.requires_grad_(not frozen)
    x, up = torch.randn(3, 200, requires_grad=True), torch.randn(3, 200)

    def gradient(create_graph, z):
        y = norm(z, z + 1)[0] if residual else norm(z)
        return torch.autograd.grad((y * up if linear else y.square()).sum(), x, create_graph=create_graph)[0]
    for z in (lambda: x, x.square):            # x itself, and what can be differentiated twice
        first = gradient(True, z())
        assert first.requires_grad
        with pytest.raises(RuntimeError, match="once only"):
            torch.autograd.grad(first.square().sum() + x.square().sum(), x)
        assert torch.equal(first, gradient(False, z()))      # once is as it is without a graph


@pytest.mark.parametrize("how", HOW)
def test_norm_gain(A, how):
    """The gain's gradient depends on x too."""
    norm = A.RMSNorm(200, checkpoint=how, device="cpu")
    x = torch.randn(3, 200, requires_grad=True)
    dgain, = torch.autograd.grad(norm(x).sum(), norm.gain, create_graph=True)
    with pytest.raises(RuntimeError, match="once only"):
        torch.autograd.grad(dgain.square().sum() + x.sum(), x)


@pytest.mark.parametrize("how", ["int8", "fp8"])
def test_norm_keeps_codes_alone(A, how):
    """What refuses a second derivative holds no memory: between the passes there are the codes, scales and row scales."""
    norm = A.RMSNorm(256, checkpoint=how, device="cpu")
    x = torch.randn(8, 256, requires_grad=True)
    kept = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: kept.append(t.untyped_storage().nbytes()) or t, lambda t: t):
        y = norm(x)
    assert sorted(kept, reverse=True)[:2] == [8 * 256, 4 * 256] and sum(kept) == 8 * 256 + 4 * 256 + 4 * 8 * 2 + 4 * 8
    y.sum().backward()
    assert x.grad is not None and norm.gain.grad is not None


@pytest.fixture()
def layers(A, monkeypatch):
    def product(x, w, ends, out, nt):
        out.data.copy_(R.grouped(x.detach(), w, ends, nt)[0])

    def grouped_gated(X, W, ends, H, *, gate_up=None, gate_up_scale=None, act):
        gu, n = R.grouped(X.detach(), W, ends, True)[0], H.shape[1]
        H.copy_(R.act(act, gu[:, :n])[0] * gu[:, n:])
        if gate_up_scale is not None:
            q, s = R.quantize(gu, gate_up.dtype)
            gate_up.copy_(q), gate_up_scale.copy_(s.view(gate_up_scale.shape))
        elif gate_up is not None:
            gate_up.copy_(gu)

    def grouped_gated_dgrad(dY, W, ends, gate_up, dgate_up, *, H=None, gate_up_scale=None, act):
        v, n = gate_up.double() if gate_up_scale is None else R.value(gate_up, gate_up_scale), H.shape[1]
        (dg, du, h), _ = R.gated_grads(act, R.grouped(dY.detach(), W, ends, False)[0], v[:, :n], v[:, n:])
        dgate_up.copy_(torch.cat([dg, du], 1)), H.copy_(h)
    steps = []
    monkeypatch.setattr(A, "grouped_gated", grouped_gated)
    monkeypatch.setattr(A, "grouped_gated_dgrad", grouped_gated_dgrad)
    monkeypatch.setattr(A, "grouped_gemm", lambda x, w, ends, y: product(x, w, ends, y, True))
    monkeypatch.setattr(A, "grouped_dgrad", lambda x, w, ends, y: product(x, w, ends, y, False))
    monkeypatch.setattr(A, "grouped_wgrad_step", lambda *a, **k: steps.append(k["step"]))
    monkeypatch.setattr(A, "block_dequantize", lambda q, s, y: y.copy_(R.value(q, s)))
    return A, steps


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("linear", [False, True])
def test_gated(layers, how, linear):
    """Its gradient depends on x through the activation, whatever arrives."""
    A, steps = layers
    torch.manual_seed(2)
    block = A.FusedGatedExperts(2, 128, 128, checkpoint=how, device="cpu")
    x, ends = torch.randn(5, 128, requires_grad=True), torch.tensor([2, 5], dtype=torch.int32)

    def gradient(create_graph, z):
        y = block(z, ends).float()
        return torch.autograd.grad((y if linear else y.square()).sum(), x, create_graph=create_graph)[0]
    for z in (lambda: x, x.square):
        first = gradient(True, z())
        assert first.requires_grad
        with pytest.raises(RuntimeError, match="once only"):
            torch.autograd.grad(first.square().sum() + x.square().sum(), x)
        assert torch.equal(first, gradient(False, z()))
    assert steps == [1, 1, 2, 2, 3, 3, 4, 4]
    # a gradient that is kept with its graph can be cleared as any other
    block(x, ends).sum().backward(create_graph=True)
    torch.optim.SGD([x], lr=1.0).zero_grad(set_to_none=False)
    assert not x.grad.any()


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("experts", [False, True])
def test_linear_layers(layers, monkeypatch, experts, how):
    """Their gradient depends on x through the arriving gradient alone: where that is constant, so is it."""
    A, steps = layers

    def linear_backward_step(x, dy, W, dx, m, v, **k):
        dx.copy_(dy.detach() @ W)
        steps.append(k["step"])
    monkeypatch.setattr(A, "linear_backward_step", linear_backward_step)
    torch.manual_seed(3)
    layer = (A.FusedExperts(2, 128, 256, checkpoint=how, device="cpu") if experts
             else A.FusedLinear(128, 256, checkpoint=how, device="cpu"))
    x, args = torch.randn(5, 128, requires_grad=True), (torch.tensor([2, 5], dtype=torch.int32),) if experts else ()

    def gradient(create_graph, linear):
        y = layer(x, *args).float()
        return torch.autograd.grad((y if linear else y.square()).sum(), x, create_graph=create_graph)[0]
    first = gradient(True, False)
    with pytest.raises(RuntimeError, match="once only"):
        torch.autograd.grad(first.square().sum() + x.square().sum(), x)
    assert torch.equal(first, gradient(False, False))
    first = gradient(True, True)
    assert torch.equal(torch.autograd.grad((first * x).sum(), x)[0], first)     # a constant gradient's penalty
    assert steps == [1, 2, 3]
