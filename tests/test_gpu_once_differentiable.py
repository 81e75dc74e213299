"""Second derivatives of the autograd layers with the library's own calls (tests/test_once_differentiable_host.py has every
combination): under create_graph the gradients are those without it, and differentiating them raises."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _name(request):
    print("[case]", request.node.name, flush=True)
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("how", [None, "int8", "fp8"])
@pytest.mark.parametrize("kind", ["norm", "linear", "experts", "gated"])
def test_layers(kind, how):
    from optimizer_step_weight_amd.autograd import FusedExperts, FusedGatedExperts, FusedLinear, RMSNorm
    ends = torch.tensor([2, 5], dtype=torch.int32, device="cuda")
    torch.manual_seed(1)
    x = torch.randn(5, 256, device="cuda").to(torch.bfloat16).requires_grad_(True)

    def gradient(create_graph):
        torch.manual_seed(2)      # the same weights: a backward pass updates them
        layer, args = {"norm": lambda: (RMSNorm(256, checkpoint=how), ()), "linear": lambda: (FusedLinear(256, 128, checkpoint=how), ()),
                       "experts": lambda: (FusedExperts(2, 256, 128, checkpoint=how), (ends,)),
                       "gated": lambda: (FusedGatedExperts(2, 256, 128, checkpoint=how), (ends,))}[kind]()
        return torch.autograd.grad(layer(x, *args).float().square().sum(), x, create_graph=create_graph)[0]
    first = gradient(True)
    assert torch.equal(first, gradient(False)) and bool(first.isfinite().all())
    with pytest.raises(RuntimeError, match="once only"):
        torch.autograd.grad(first.float().square().sum() + x.float().square().sum(), x)
