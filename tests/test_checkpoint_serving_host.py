"""Layers with `checkpoint` on the CPU, with stand-ins for the library's calls: codes are made only where a backward pass
will read them."""
import pytest
import torch


@pytest.fixture()
def made(monkeypatch):
    from optimizer_step_weight_amd import autograd
    made = []
    monkeypatch.setattr(autograd, "rmsnorm", lambda x, gain, y, *, residual=None, h=None, rstd=None, eps: (
        y.zero_(), rstd.zero_(), None if h is None else h.zero_()))
    monkeypatch.setattr(autograd, "grouped_gemm", lambda x, w, ends, y: y.zero_())
    monkeypatch.setattr(autograd, "block_quantize", lambda x, q, s: made.append(tuple(x.shape)))
    return autograd, made


def layers(A, how):
    ends = torch.tensor([2, 5], dtype=torch.int32)
    norm = A.RMSNorm(128, checkpoint=how, device="cpu")
    return [(A.FusedLinear(128, 256, checkpoint=how, device="cpu"), ()), (A.FusedExperts(2, 128, 256, checkpoint=how, device="cpu"), (ends,)),
            (norm, ()), (norm, (torch.ones(5, 128),))]


@pytest.mark.parametrize("how", ["int8", "fp8"])
@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_no_codes_without_gradients(made, how, mode):
    A, made = made
    for layer, args in layers(A, how):
        for x in (torch.ones(5, 128), torch.ones(5, 128, requires_grad=True)):
            layer(x, *args)
            assert made.pop() == (5, 128) and not made       # for a backward pass
            with mode():
                layer(x, *args)
            assert not made


def test_no_codes_where_nothing_needs_a_gradient(made):
    A, made = made
    norm = A.RMSNorm(128, checkpoint="int8", device="cpu").requires_grad_(False)
    norm(torch.ones(5, 128))
    assert not made
    norm(torch.ones(5, 128, requires_grad=True))
    assert made == [(5, 128)]
