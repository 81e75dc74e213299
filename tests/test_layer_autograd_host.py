"""The autograd layers around the experts on the CPU, the library's calls replaced by plain torch ones that
write into the tensors they are given, as the library does."""
import pytest
import torch

from tests import layer_ref as R


@pytest.fixture()
def A(monkeypatch):
    from optimizer_step_weight_amd import autograd

    def rows(t):
        assert t.data_ptr() % 16 == 0 and t.is_contiguous()     # what the library asks of every tensor
        return t.detach().double()

    def rmsnorm(x, gain, y, *, residual=None, h=None, rstd=None, eps):
        for t in (y, rstd, h):
            assert t is None or t.data_ptr() % 4 == 0
        s = x if residual is None else (x.float() + residual.float()).to(x.dtype)
        out, r = R.norm(rows(s), rows(gain), eps)
        rows(x), residual is None or rows(residual)
        rows(y), y.data.copy_(out), rstd.data.copy_(r)
        if h is not None:
            h.data.copy_(s)

    def rmsnorm_backward(dy, h, gain, rstd, dx, dgain=None, *, dh=None):
        gx, gg = R.norm_grads(rows(dy), rows(h), rows(gain), rstd.detach().double(), None if dh is None else rows(dh))
        dx.data.copy_(gx)
        if dgain is not None:
            dgain.data.copy_(gg)
    monkeypatch.setattr(autograd, "rmsnorm", rmsnorm)
    monkeypatch.setattr(autograd, "rmsnorm_backward", rmsnorm_backward)
    return autograd


@pytest.mark.parametrize("residual", [False, True])
def test_norm_second_derivatives_are_refused(A, residual):
    """The gradient comes out of the library without a graph: to differentiate it again raises."""
    norm = A.RMSNorm(16, device="cpu")
    x = torch.randn(3, 16, requires_grad=True)

    def gradient(create_graph):
        z = x.square()                 # differentiable twice, so that the whole keeps a graph
        y = norm(z, z + 1)[0] if residual else norm(z)
        return torch.autograd.grad(y.square().sum(), x, create_graph=create_graph)[0]
    first = gradient(True)
    with pytest.raises(RuntimeError, match="once only"):
        torch.autograd.grad(first.square().sum(), x)
    assert torch.equal(first, gradient(False))     # once is as it was


@pytest.mark.parametrize("use", ["y", "h", "both"])
@pytest.mark.parametrize("frozen", [False, True])
def test_norm_gradients_of_either_output(A, use, frozen):
    g = torch.Generator().manual_seed(1)
    norm = A.RMSNorm(24, eps=1e-3, device="cpu")
    norm.gain.requires_grad_(not frozen)
    x, r, up, uh = (torch.randn(5, 24, generator=g) for _ in range(4))
    x.requires_grad_(True), r.requires_grad_(True)
    y, h = norm(x, r)
    loss = (y * up).sum() * (use != "h") + (h * uh).sum() * (use != "y")
    want = torch.autograd.grad(loss, [x, r] + ([] if frozen or use == "h" else [norm.gain]))
    x2, r2, w2 = x.detach().double().requires_grad_(True), r.detach().double().requires_grad_(True), torch.ones(24).double().requires_grad_(True)
    y2 = R.norm(x2 + r2, w2, 1e-3)[0]
    loss2 = (y2 * up).sum() * (use != "h") + ((x2 + r2) * uh).sum() * (use != "y")
    exact = torch.autograd.grad(loss2, [x2, r2] + ([] if frozen or use == "h" else [w2]))
    for a, b in zip(want, exact):
        assert torch.allclose(a.double(), b, rtol=1e-5, atol=1e-5)


def misplaced(t):
    """The same values in a contiguous tensor whose data is not 16-byte aligned."""
    out = torch.empty(t.numel() + 1, dtype=t.dtype)[1:].view(t.shape)
    assert out.is_contiguous() and out.data_ptr() % 16 != 0
    return out.copy_(t.detach())


@pytest.mark.parametrize("where", ["x", "residual", "gain", "dy", "dh", "column slice"])
def test_norm_of_views_that_are_not_aligned(A, where):
    g = torch.Generator().manual_seed(3)
    norm = A.RMSNorm(15, device="cpu")
    x, r, dy, dh = (torch.randn(4, 15, generator=g) for _ in range(4))

    def run(x, r, dy, dh):
        x, r = x.detach().requires_grad_(True), r.detach().requires_grad_(True)
        norm.gain.grad = None
        y, h = norm(x, r)
        torch.autograd.backward([y, h], [dy, dh])
        return y, h, x.grad, r.grad, norm.gain.grad
    want = run(x, r, dy, dh)
    if where == "gain":
        norm.gain = torch.nn.Parameter(misplaced(norm.gain))
        assert norm.gain.data_ptr() % 16 != 0
    moved = [misplaced(t) if n == where else t for n, t in (("x", x), ("residual", r), ("dy", dy), ("dh", dh))]
    if where == "column slice":   # neither contiguous nor aligned
        moved = [torch.cat([t[:, :1], t], 1)[:, 1:] for t in moved]
    assert all(torch.equal(a, b) for a, b in zip(run(*moved), want))


@pytest.mark.parametrize("layer", ["experts", "linear"])
def test_trained_layers_of_views_that_are_not_aligned(A, monkeypatch, layer):
    """Inputs and incoming gradients are copied where the library could not take them."""
    seen = []

    def take(*tensors, **kw):
        for t in tensors:
            if isinstance(t, torch.Tensor) and t.dtype == torch.bfloat16:
                assert t.data_ptr() % 16 == 0 and t.is_contiguous()
        seen.append(len(tensors))
    for name in ("grouped_gemm", "grouped_dgrad", "grouped_wgrad_step", "linear_backward_step"):
        monkeypatch.setattr(A, name, take)
    BF = torch.bfloat16
    x, dy = torch.randn(6, 128).to(BF), torch.randn(6, 256).to(BF)
    mod = A.FusedExperts(2, 128, 256, device="cpu") if layer == "experts" else A.FusedLinear(128, 256, device="cpu")
    xm = misplaced(x).requires_grad_(True)
    y = mod(xm, torch.tensor([2, 6], dtype=torch.int32)) if layer == "experts" else mod(xm)
    y.backward(misplaced(dy))
    assert len(seen) == (3 if layer == "experts" else 1) and xm.grad.shape == x.shape
