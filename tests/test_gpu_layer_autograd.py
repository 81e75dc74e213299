"""The autograd layers around the experts (optimizer_step_weight_amd.autograd.RMSNorm, FusedExperts)
and the example that trains with them: gradients against the formulas and against differences, the
weights' update against the library's calls, and a loss that falls."""
import importlib.util
import os

import pytest
import torch

from tests import layer_ref as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    import optimizer_step_weight_amd as forge
    forge.device_check(0)
    return forge


@pytest.fixture(autouse=True)
def _name(request):
    print("[case]", request.node.name, flush=True)
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("residual", [True, False])
def test_norm_gradients_against_differences(lib, residual):
    """Central differences of the 64-bit definition along random directions."""
    from optimizer_step_weight_amd.autograd import RMSNorm
    T, D, eps = 5, 264, 1e-6
    g = torch.Generator().manual_seed(3)
    x, r = torch.randn(T, D, generator=g), torch.randn(T, D, generator=g)
    up, uh = torch.randn(T, D, generator=g), torch.randn(T, D, generator=g)
    norm = RMSNorm(D, eps=eps)
    with torch.no_grad():
        norm.gain.copy_(1 + 0.3 * torch.randn(D, generator=g))
    xd, rd = x.cuda().requires_grad_(True), r.cuda().requires_grad_(True)
    if residual:
        y, h = norm(xd, rd)
        ((y * up.cuda()).sum() + (h * uh.cuda()).sum()).backward()
        assert torch.equal(xd.grad, rd.grad)
    else:
        (norm(xd) * up.cuda()).sum().backward()

    def value(a, w):
        h = a + (r.double() if residual else 0.0)
        y, _ = R.norm(h, w, eps)
        return (y * up.double()).sum() + ((h * uh.double()).sum() if residual else 0.0)

    a, w, step = x.double(), norm.gain.detach().cpu().double(), 1e-5
    for seed in range(4):
        g = torch.Generator().manual_seed(50 + seed)
        da, dw = torch.randn(T, D, generator=g).double(), torch.randn(D, generator=g).double()
        for base, grad, d, f in ((a, xd.grad, da, lambda t: value(t, w)), (w, norm.gain.grad, dw, lambda t: value(a, t))):
            want = (f(base + step * d) - f(base - step * d)) / (2 * step)
            got = (grad.cpu().double() * d).sum()
            # fp32 gradients: a few dozen roundings of each term; the difference itself is off by the
            # square of its step and by 2^-53 / step of the value
            scale = (grad.cpu().double() * d).abs().sum() + 1.0
            assert abs(got - want) <= 64 * R.U * scale + 1e-7 * scale, (float(got), float(want))


def test_experts_backward_is_the_library_calls(lib):
    from optimizer_step_weight_amd.autograd import FusedExperts
    E, K, N, T = 3, 256, 384, 200
    g = torch.Generator().manual_seed(1)
    W = (0.05 * torch.randn(E, N, K, generator=g)).to(BF).cuda()
    x, dy = torch.randn(T, K, generator=g).to(BF).cuda(), (0.1 * torch.randn(T, N, generator=g)).to(BF).cuda()
    ends = torch.tensor([20, 20, 190], dtype=torch.int32, device="cuda")
    layer = FusedExperts(E, K, N, hyper={"lr": 1e-2}, seed=5, weight=W.clone())
    xi = x.clone().requires_grad_(True)
    y = layer(xi, ends)
    Y, dX = torch.empty_like(dy), torch.empty_like(x)
    lib.grouped_gemm(x, W, ends, Y)
    assert torch.equal(y, Y)
    y.backward(dy)
    lib.grouped_dgrad(dy, W, ends, dX)
    assert torch.equal(xi.grad, dX)
    W1, m, v = W.clone(), torch.zeros(E, N, K, device="cuda"), torch.zeros(E, N, K, device="cuda")
    lib.grouped_wgrad_step(x, dy, ends, W1, m, v, opt="adamw", hyper={"lr": 1e-2}, step=1, seed=5)
    assert torch.equal(layer.weight, W1) and torch.equal(layer.m, m) and torch.equal(layer.v, v)
    assert layer.step_count == 1 and not torch.equal(W1, W)
    with pytest.raises(ValueError):
        layer(x[:, :128], ends)
    with pytest.raises(ValueError):
        layer(x, ends[:2])


def test_example_trains(lib):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses = mod.train(30)
    assert all(x == x for x in losses) and sum(losses[-5:]) < 0.7 * sum(losses[:5]), losses
