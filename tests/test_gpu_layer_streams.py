"""Buffers that the binding owns, when the work runs on another stream than the current one: they are not
handed to other work before that stream is done with them."""
import pytest
import torch

from tests import layer_ref as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
BUSY = 50_000_000      # clock ticks that keep a stream busy: some tens of milliseconds


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


def fill_new_blocks(size, count=4):
    """New blocks of `size` bytes on the current stream, written at once."""
    return [torch.full((size // 4,), float("nan"), device="cuda") for _ in range(count)]


def test_norm_backward_workspace_belongs_to_the_stream(lib):
    T, D = 700, 1024
    g = torch.Generator().manual_seed(1)
    h, dy, gain = torch.randn(T, D, generator=g).to(BF), torch.randn(T, D, generator=g).to(BF), torch.ones(D)
    rstd = R.norm(h, gain, 1e-6)[1].float()
    h, dy, gain, rstd = (t.cuda() for t in (h, dy, gain, rstd))
    size = 4 * lib.rmsnorm_backward_workspace(T, D).numel()
    dx, dgain, dx1, dgain1 = torch.empty_like(h), torch.empty(D, device="cuda"), torch.empty_like(h), torch.empty(D, device="cuda")
    lib.rmsnorm_backward(dy, h, gain, rstd, dx, dgain)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
    lib.rmsnorm_backward(dy, h, gain, rstd, dx1, dgain1, stream=s.cuda_stream)
    kept = fill_new_blocks(size)
    torch.cuda.synchronize()
    assert torch.equal(dx, dx1) and torch.equal(dgain, dgain1)
    assert all(torch.isnan(t).all() for t in kept)
    # the default stream by its address
    lib.rmsnorm_backward(dy, h, gain, rstd, dx1.zero_(), dgain1.zero_(), stream=0)
    assert torch.equal(dx, dx1) and torch.equal(dgain, dgain1)


def test_one_launch_backward_workspace_belongs_to_the_stream(lib):
    T, N, K = 256, 256, 384
    g = torch.Generator().manual_seed(2)
    X, dY = torch.randn(T, K, generator=g).to(BF).cuda(), (0.1 * torch.randn(T, N, generator=g)).to(BF).cuda()
    W0 = (0.05 * torch.randn(N, K, generator=g)).to(BF).cuda()
    size = lib.backward_workspace_bytes(K)
    s, out = torch.cuda.Stream(), []
    for stream in (None, s.cuda_stream, 0):
        W, m, v, dX = W0.clone(), torch.zeros(N, K, device="cuda"), torch.zeros(N, K, device="cuda"), torch.empty_like(X)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(BUSY)
        lib.linear_backward_step_fused(X, dY, W, dX, m, v, step=1, seed=3, stream=stream)   # the workspace is dropped
        kept = fill_new_blocks(size)
        torch.cuda.synchronize()
        out.append((W, m, v, dX))
        assert all(torch.isnan(t).all() for t in kept)
    for other in out[1:]:
        assert all(torch.equal(a, b) for a, b in zip(out[0], other))


def busy_step(lib, s):
    """A plan and its tensors, with a step queued on s behind other work."""
    w, g = [torch.zeros(300, device="cuda"), torch.zeros(5000, device="cuda")], None
    g = [torch.ones_like(t) for t in w]
    plan = lib.MultiStep(w, g, opt="sgd")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
    plan.step(step=1, hyper={"lr": 1.0}, stream=s.cuda_stream)
    return plan, w, g


def test_table_outlives_a_step_on_another_stream(lib):
    """Both after set_grads and after the plan is gone, also where the step's stream is the current one."""
    s = torch.cuda.Stream()
    plan, w, g = busy_step(lib, s)
    size = plan._table.numel()
    plan.set_grads([torch.full_like(t, 2.0) for t in w])
    kept = fill_new_blocks(size)
    torch.cuda.synchronize()
    assert all(bool((t == -1.0).all()) for t in w)
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
        plan.step(step=2, hyper={"lr": 1.0})
    del plan
    kept += fill_new_blocks(size)
    torch.cuda.synchronize()
    assert all(bool((t == -3.0).all()) for t in w)
    plan, w, g = busy_step(lib, s)
    del plan
    kept += fill_new_blocks(size)
    torch.cuda.synchronize()
    assert all(bool((t == -1.0).all()) for t in w) and all(torch.isnan(t).all() for t in kept)


@pytest.mark.parametrize("home", [False, True])
def test_captured_step_keeps_its_table_and_gradients(lib, home):
    """A graph replays with the gradients of its capture, whatever set_grads did since."""
    s = torch.cuda.Stream()
    w, graph = [torch.zeros(300, device="cuda"), torch.zeros(5000, device="cuda")], torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s) if home else torch.cuda.stream(torch.cuda.current_stream()):
        plan = lib.MultiStep(w, [torch.ones_like(t) for t in w], opt="sgd")
        size = plan._table.numel()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        plan.step(step=1, hyper={"lr": 1.0})
        plan.step(step=1, hyper={"lr": 1.0})
    total = 0.0
    for i in range(3):
        with torch.cuda.stream(s):
            plan.set_grads([torch.full_like(t, 4.0) for t in w])
            kept = fill_new_blocks(size) + [torch.full_like(t, float("nan")) for t in w]
        torch.cuda.synchronize()
        graph.replay()
        plan.step(step=2, hyper={"lr": 1.0})
        torch.cuda.synchronize()
        total += 2.0 + 4.0
        assert all(bool((t == -total).all()) for t in w) and all(torch.isnan(t).all() for t in kept)
    assert len(plan._captured) == 1
