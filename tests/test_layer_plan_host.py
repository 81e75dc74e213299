"""MultiStep's host side, no GPU needed: the plan packs host tensors here (their addresses are never used),
so that its table, its state after a refusal and its hyper-parameters can be looked at."""
import ctypes
import os

import pytest
import torch


@pytest.fixture()
def f(monkeypatch):
    import optimizer_step_weight_amd as forge
    if not os.path.exists(forge.LIB_PATH):
        from optimizer_step_weight_amd import _build
        _build.build(verbose=False)
    from optimizer_step_weight_amd import layer
    monkeypatch.setattr(layer, "_device", lambda t, what: -1)     # where a host tensor says it is
    monkeypatch.setattr(layer, "_current_device", lambda: -1)
    monkeypatch.setattr(layer, "_stream", lambda stream, dev: 0)
    monkeypatch.setattr(layer, "_capturing", lambda: False)
    return forge


def plan_of(f, sizes=(5, 4096, 70_000)):
    W, g, m, v = ([torch.zeros(n) for n in sizes] for _ in range(4))
    return f.MultiStep(W, g, m, v, opt="adamw"), W, g


def state(plan):
    info = plan._info
    return bytes(ctypes.string_at(ctypes.addressof(info), ctypes.sizeof(info))), plan._table.clone(), plan._lists["g"]


@pytest.mark.parametrize("bad", ["type", "size", "count", "alias", "alignment", "none"])
def test_refused_gradients_leave_the_plan_as_it_was(f, bad):
    plan, W, g = plan_of(f)
    info, table, grads = state(plan)
    new = [torch.ones_like(t) for t in g]
    if bad == "type":
        new[2] = new[2].to(torch.float16)
    elif bad == "size":
        new[1] = new[1][:-1]
    elif bad == "count":
        new = new[:2]
    elif bad == "alias":
        new[2] = W[2]
    elif bad == "alignment":
        new[1] = torch.ones(4097)[1:]
    else:
        new[0] = None
    with pytest.raises((ValueError, TypeError, AttributeError, f.ForgeError)):
        plan.set_grads(new)
    after = state(plan)
    assert after[0] == info and torch.equal(after[1], table)
    assert len(after[2]) == len(grads) and all(a is b for a, b in zip(after[2], grads))


def test_gradients_taken(f):
    plan, _, g = plan_of(f)
    _, table, _ = state(plan)
    new = [torch.ones_like(t) for t in g]
    plan.set_grads(new)
    info, other, grads = state(plan)
    assert not torch.equal(table, other) and all(a is b for a, b in zip(grads, new))
    at = [int.from_bytes(bytes(other[72 * i + 8:72 * i + 16].tolist()), "little") for i in range(3)]
    assert at == [t.data_ptr() for t in new]


def steps(f, plan, monkeypatch):
    """Calls of step() with the device's call replaced: the learning rates that it would be given."""
    from optimizer_step_weight_amd import layer
    seen = []

    class Lib:
        @staticmethod
        def forge_multi_step(info, table, hypers, n, *rest):
            seen.append([round(hypers[i].lr, 6) for i in range(n)])
            return 0
    monkeypatch.setattr(layer, "_lib", lambda: Lib)

    def call(hyper):
        plan.step(step=1, hyper=hyper)
        return seen[-1]
    return call


def test_hyper_parameters_of_a_failed_call_are_not_used(f, monkeypatch):
    plan, _, _ = plan_of(f)
    call = steps(f, plan, monkeypatch)
    a, b = {"lr": 1.0}, {"lr": 2.0}
    assert call([a, b]) == [1.0, 2.0]
    with pytest.raises(TypeError):
        call([{"lr": 9.0}, {"lr": "fast"}])
    assert call([a, b]) == [1.0, 2.0]
    assert call([b, a]) == [2.0, 1.0] and call(a) == [1.0] and call([a, b]) == [1.0, 2.0]


@pytest.mark.parametrize("kind", ["tensor", "array", "object"])
def test_hyper_parameters_changed_in_place_are_read_again(f, monkeypatch, kind):
    import types

    import numpy as np
    plan, _, _ = plan_of(f)
    call = steps(f, plan, monkeypatch)
    lr = torch.tensor(1.0) if kind == "tensor" else np.array(1.0)
    h = types.SimpleNamespace(lr=1.0) if kind == "object" else {"lr": lr}
    assert call(h) == [1.0]
    if kind == "object":
        h.lr = 3.0
    else:
        lr[...] = 3.0
    assert call(h) == [3.0]
    d = {"lr": 0.5}
    assert call(d) == [0.5]
    d["lr"] = 0.25
    assert call(d) == [0.25]


def test_host_calls_need_no_torch():
    """Versions, scalars and refusals of the C ABI in a process that has no torch."""
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ("import sys; sys.modules['torch'] = None\n"
            "import optimizer_step_weight_amd as f\n"
            "assert f.version() > 0 and f.build_id() and f.step_scalars('adamw', {'lr': 0.5}, 1)['lr'] == 0.5\n"
            "assert f._lib().forge_rmsnorm(None, None, None, 0.0, None, None, 0, None, None, None) == 1 and f.last_error()\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
