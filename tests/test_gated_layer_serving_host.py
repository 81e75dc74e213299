"""FusedGatedExperts without gradients on the CPU, with stand-ins for the library's calls."""
import pytest
import torch
import torch.autograd.forward_ad as fwd


@pytest.fixture()
def A(monkeypatch):
    from optimizer_step_weight_amd import autograd
    kept = []

    def grouped_gated(X, W, ends, H, *, gate_up=None, gate_up_scale=None, act):
        kept.append(gate_up)
        H.zero_()
    monkeypatch.setattr(autograd, "grouped_gated", grouped_gated)
    monkeypatch.setattr(autograd, "grouped_gemm", lambda X, W, ends, Y: Y.zero_())
    monkeypatch.setattr(autograd, "block_quantize", lambda *a: kept.append(a))
    return autograd, kept


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode, torch.enable_grad])
@pytest.mark.parametrize("how", [None, "int8"])
def test_forward_mode_raises(A, mode, how):
    """no_grad does not end forward-mode differentiation: an input with a tangent is refused, not answered without one."""
    A, _ = A
    block = A.FusedGatedExperts(1, 128, 128, checkpoint=how, device="cpu")
    x = torch.randn(3, 128)
    if mode is torch.inference_mode:
        with mode():
            assert block(x).shape == (3, 128)   # a tangent cannot be made there
        return
    with fwd.dual_level(), mode():
        for z in (x, x.to(torch.bfloat16)):
            with pytest.raises(RuntimeError, match="forward"):
                block(fwd.make_dual(z, torch.ones_like(z)))
        block(x)                                # the others are answered


def test_nothing_is_kept(A):
    A, kept = A
    block = A.FusedGatedExperts(1, 128, 128, checkpoint="int8", device="cpu")
    with torch.no_grad():
        y = block(torch.randn(2, 3, 128, requires_grad=True))
    assert kept == [None] and not y.requires_grad and y.shape == (2, 3, 128)
