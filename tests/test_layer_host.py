"""Host side of include/forge_layer.h, no GPU needed: refusals with their statuses (fake,
never-dereferenced addresses), the packed table of the step over many tensors, the binding's own
checks, and the norm's gradient formula against differences in 64 bits."""
import ctypes
import os

import pytest
import torch

from tests import layer_ref as R


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


def test_rmsnorm_refusals(f):
    T, D = 5, 384
    ok = dict(x=t(f, 0, T, D), res=t(f, 1, T, D), gain=t(f, 2, 1, D, f.F32), eps=1e-6, h=t(f, 3, T, D),
              y=t(f, 4, T, D, f.FP8_E4M3, scale=FAKE + 5 * GB), mode=0, rstd=FAKE + 6 * GB, amax=FAKE + 7 * GB)

    def call(**kw):
        a = dict(ok, **kw)
        return f._lib().forge_rmsnorm(ref(a["x"]), ref(a["res"]), ref(a["gain"]), a["eps"], ref(a["h"]), ref(a["y"]),
                                      a["mode"], a["rstd"], a["amax"], None)
    cases = [
        (dict(x=None), ARG), (dict(gain=None), ARG), (dict(y=None), ARG),
        (dict(x=t(f, 0, T, D, f.FP8_E4M3)), DTYPE), (dict(x=t(f, 0, T, 0), gain=t(f, 2, 1, 0)), SHAPE),
        (dict(res=None), ARG), (dict(h=None), ARG), (dict(res=t(f, 1, T, D, f.F32)), DTYPE),
        (dict(h=t(f, 3, T + 1, D)), SHAPE), (dict(gain=t(f, 2, 1, D - 1)), SHAPE), (dict(gain=t(f, 2, T, D)), SHAPE),
        (dict(gain=t(f, 2, 1, D, f.I8_B64)), DTYPE), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
        (dict(eps=float("inf")), ARG), (dict(mode=2), ARG), (dict(y=t(f, 4, T, D, f.FP8_E4M3)), ARG),
        (dict(y=t(f, 4, T, D, f.FP8_E4M3, scale=FAKE + 2)), LAYOUT), (dict(y=t(f, 4, T, D, f.I8_B64)), DTYPE),
        (dict(y=t(f, 4, T, D - 1, f.BF16)), SHAPE), (dict(x=t(f, 0, T, D, off=8)), LAYOUT),
        (dict(x=t(f, 0, T, D, ld=D + 8)), LAYOUT), (dict(rstd=FAKE + 6 * GB + 2), LAYOUT),
        (dict(amax=FAKE + 1), LAYOUT), (dict(y=t(f, 0, T, D)), ALIAS), (dict(h=t(f, 0, T, D, off=16)), ALIAS),
        (dict(h=t(f, 4, T, D)), ALIAS), (dict(rstd=FAKE + 2 * GB), ALIAS), (dict(amax=FAKE + 6 * GB + 4), ALIAS),
        (dict(x=t(f, 0, -1, D)), SHAPE), (dict(x=t(f, 0, 1 << 31, D)), SHAPE),
    ]
    for kw, want in cases:
        assert call(**kw) == want, (kw, f.last_error())
        assert f.last_error()
    empty = dict(x=t(f, 0, 0, D), res=t(f, 1, 0, D), h=t(f, 3, 0, D), y=t(f, 4, 0, D))
    assert call(**empty) == 0, f.last_error()
    assert call(**dict(empty, h=t(f, 0, 0, D))) == 0


def test_rmsnorm_backward_refusals(f):
    T, D = 5, 384
    need = f._lib().forge_rmsnorm_backward_workspace_bytes(T, D)
    assert need >= 4 * D and f._lib().forge_rmsnorm_backward_workspace_bytes(-1, 4) == -1
    ok = dict(dy=t(f, 0, T, D), dh=t(f, 1, T, D), h=t(f, 2, T, D), gain=t(f, 3, 1, D, f.F32), rstd=FAKE + 4 * GB,
              dx=t(f, 5, T, D), dgain=t(f, 6, 1, D, f.F32), ws=FAKE + 7 * GB, n=need)

    def call(**kw):
        a = dict(ok, **kw)
        return f._lib().forge_rmsnorm_backward(ref(a["dy"]), ref(a["dh"]), ref(a["h"]), ref(a["gain"]), a["rstd"],
                                               ref(a["dx"]), ref(a["dgain"]), a["ws"], a["n"], None)
    for kw, want in [
        (dict(dy=None), ARG), (dict(h=None), ARG), (dict(dx=None), ARG), (dict(gain=None), ARG), (dict(rstd=None), ARG),
        (dict(h=t(f, 2, T, D, f.F32)), DTYPE), (dict(dh=t(f, 1, T, D, f.F32)), DTYPE), (dict(dx=t(f, 5, T + 1, D)), SHAPE),
        (dict(dgain=t(f, 6, 1, D)), DTYPE), (dict(dgain=t(f, 6, 1, D + 1, f.F32)), SHAPE), (dict(ws=None), ARG),
        (dict(n=need - 1), ARG), (dict(ws=FAKE + 7 * GB + 4), LAYOUT), (dict(ws=FAKE + 2 * GB), ALIAS),
        (dict(dx=t(f, 2, T, D)), ALIAS), (dict(dx=t(f, 0, T, D, off=16)), ALIAS), (dict(dgain=t(f, 3, 1, D, f.F32)), ALIAS),
    ]:
        assert call(**kw) == want, (kw, f.last_error())
    z = lambda s: t(f, s, 0, D)  # noqa: E731
    assert call(dy=z(0), dh=z(1), h=z(2), dx=z(5), dgain=None, ws=None, n=0) == 0
    assert call(dy=z(0), dh=None, h=z(2), dx=z(0), dgain=None, ws=None, n=0) == 0   # in place


def test_grouped_refusals(f):
    T, N, K, E = 70, 256, 384, 3
    X, dY, W = t(f, 0, T, K), t(f, 1, T, N), t(f, 2, E * N, K)
    Y, dX, dW, ends = t(f, 3, T, N), t(f, 4, T, K), t(f, 5, E * N, K, f.F32), FAKE + 6 * GB
    L = f._lib()
    for a, want in [
        ((None, W, ends, E, Y), ARG), ((X, W, None, E, Y), ARG), ((X, W, ends, 0, Y), ARG), ((X, W, ends, 4097, Y), ARG),
        ((X, W, ends + 2, E, Y), LAYOUT), ((X, W, ends, 2, Y), SHAPE), ((X, t(f, 2, E * N, K, f.F32), ends, E, Y), DTYPE),
        ((X, W, ends, E, t(f, 3, T, N, f.F32)), DTYPE), ((t(f, 0, T, 64), t(f, 2, E * N, 64), ends, E, Y), SHAPE),
        ((X, W, ends, E, t(f, 3, T - 1, N)), SHAPE), ((X, W, ends, E, t(f, 0, T, N)), ALIAS),
        ((X, W, FAKE + 3 * GB + 8, E, Y), ALIAS),
        ((t(f, 0, T, K, f.FP8_E4M3), t(f, 2, E * N, K, f.FP8_E4M3), ends, E, Y), ARG),
        ((t(f, 0, T, 1 << 21), t(f, 2, E * N, 1 << 21), ends, E, Y), SHAPE),
        ((t(f, 0, T, 1 << 20), t(f, 2, E * 2048, 1 << 20), ends, E, t(f, 3, T, 2048)), SHAPE),
    ]:
        x, w, at, n, y = a
        assert L.forge_grouped_gemm(ref(x), ref(w), at, n, ref(y), None) == want, (a, f.last_error())
    assert L.forge_grouped_gemm(r(t(f, 0, 0, K)), r(W), ends, E, r(t(f, 3, 0, N)), None) == 0
    for a, want in [((dY, W, ends, E, None), ARG), ((dY, W, ends, E, t(f, 4, T, K + 128)), SHAPE),
                    ((t(f, 1, T, N, f.FP8_E4M3), t(f, 2, E * N, K, f.FP8_E4M3), ends, E, dX), DTYPE),
                    ((dY, W, ends, E, t(f, 2, T, K)), ALIAS)]:
        x, w, at, n, y = a
        assert L.forge_grouped_dgrad(ref(x), ref(w), at, n, ref(y), None) == want, (a, f.last_error())
    for a, want in [((X, t(f, 1, T + 1, N), ends, E, dW), SHAPE), ((X, dY, ends, E, t(f, 5, E * N, K)), DTYPE),
                    ((X, dY, ends, E, t(f, 5, N, K, f.F32)), SHAPE), ((t(f, 0, T, K, f.F32), dY, ends, E, dW), DTYPE),
                    ((X, dY, ends, E, t(f, 1, E * N, K, f.F32)), ALIAS),
                    ((t(f, 0, 1 << 24, K), t(f, 1, 1 << 24, N), ends, E, dW), SHAPE)]:
        x, d, at, n, w = a
        assert L.forge_grouped_wgrad(ref(x), ref(d), at, n, ref(w), None) == want, (a, f.last_error())
    m, v, h = t(f, 7, E * N, K, f.F32), t(f, 8, E * N, K, f.F32), f._hyper({})
    for a, kw, want in [((X, dY, W, None, v), {}, ARG), ((X, dY, W, m, v), dict(step=0), ARG),
                        ((X, dY, t(f, 2, E * N, K, f.F32), m, v), {}, DTYPE), ((X, dY, t(f, 2, N, K), m, v), {}, SHAPE),
                        ((X, dY, t(f, 0, E * N, K), m, v), {}, ALIAS), ((X, dY, W, m, t(f, 7, E * N, K, f.F32)), {}, ALIAS),
                        ((X, dY, W, m, v), dict(opt=8), ARG), ((X, dY, W, t(f, 7, E * N, K, f.I8_B64), v), {}, ARG)]:
        x, d, w, mm, vv = a
        assert L.forge_grouped_wgrad_step(ref(x), ref(d), ends, E, ref(w), ref(mm), ref(vv), r(h), kw.get("opt", 0),
                                          kw.get("step", 1), 0, None, None) == want, (a, kw, f.last_error())


def _entry(f, i, n, **kw):
    from optimizer_step_weight_amd.layer import _MultiTensor
    base = FAKE + i * GB
    e = _MultiTensor(base, base + (64 << 20), base + (128 << 20), base + (192 << 20), None, None, n, 7, f.F32, f.BF16, 0, 0)
    for k, v in kw.items():
        setattr(e, k, v)
    return e


def _pack(f, entries, opt=0, md=None, vd=None, short=0):
    from optimizer_step_weight_amd.layer import _MultiInfo, _MultiTensor
    a = (_MultiTensor * len(entries))(*entries)
    L = f._lib()
    n = L.forge_multi_table_bytes(a, len(entries))
    buf, info = ctypes.create_string_buffer(max(n, 1)), _MultiInfo()
    st = L.forge_multi_pack(a, len(entries), opt, f.F32 if md is None else md, f.F32 if vd is None else vd, buf,
                            n - short, r(info))
    return st, info, bytes(buf.raw[:max(n, 0)])


def test_multi_pack_table(f):
    """The table of a few tensors: chunk counts, and each chunk's owner."""
    sizes = [1, 0, 4096, 4097, 300_000]
    st, info, raw = _pack(f, [_entry(f, i, n, group=i % 3) for i, n in enumerate(sizes)])
    assert st == 0, f.last_error()
    chunks = [-(-n // 4096) for n in sizes]
    assert (info.tensors, info.groups, info.chunks, info.bytes) == (5, 3, sum(chunks), len(raw))
    owner = [int.from_bytes(raw[5 * 72 + 4 * c:5 * 72 + 4 * c + 4], "little") for c in range(info.chunks)]
    assert owner == [i for i, c in enumerate(chunks) for _ in range(c)]
    assert [int.from_bytes(raw[72 * i + 60:72 * i + 64], "little") for i in range(5)] == [0, 1, 1, 2, 4]
    assert _pack(f, [])[0] == 0


def test_multi_refusals(f):
    n = 1000
    I8, U8 = f.I8_B64, f.U8_B64
    S = FAKE + 90 * GB
    for entries, kw, want in [
        ([_entry(f, 0, n, W=None)], {}, ARG), ([_entry(f, 0, n, g=None)], {}, ARG), ([_entry(f, 0, n, m=None)], {}, ARG),
        ([_entry(f, 0, n, v=None)], {}, ARG), ([_entry(f, 0, n)], dict(opt=6), ARG), ([_entry(f, 0, n)], dict(opt=9), ARG),
        ([_entry(f, 0, n, group=8)], {}, ARG), ([_entry(f, 0, n, reserved=1)], {}, ARG),
        ([_entry(f, 0, n, w_dtype=f.I8_B64)], {}, DTYPE), ([_entry(f, 0, n, g_dtype=f.FP8_E4M3)], {}, DTYPE),
        ([_entry(f, 0, n, W=FAKE + 4)], {}, LAYOUT), ([_entry(f, 0, -1)], {}, SHAPE), ([_entry(f, 0, 1 << 32)], {}, SHAPE),
        ([_entry(f, 0, n), _entry(f, 0, n)], {}, ALIAS), ([_entry(f, 0, n), _entry(f, 1, n, W=FAKE + 3200)], {}, ALIAS),
        ([_entry(f, 0, n, g=FAKE)], {}, ALIAS), ([_entry(f, 0, n)], dict(md=I8, vd=f.F32), DTYPE),
        ([_entry(f, 0, n)], dict(md=I8, vd=f.U8DYN_B64), DTYPE), ([_entry(f, 0, n)], dict(md=I8, vd=U8), ARG),
        ([_entry(f, 0, n, m_scale=S, v_scale=S + 6)], dict(md=I8, vd=U8), LAYOUT),
        ([_entry(f, 0, n, m_scale=S, v_scale=S + 60)], dict(md=I8, vd=U8), ALIAS),
        ([_entry(f, 0, n, m_scale=S)], {}, ARG), ([_entry(f, 0, n)], dict(short=1), ARG),
    ]:
        assert _pack(f, entries, **kw)[0] == want, (kw, f.last_error())
    # shared gradients are read only: allowed
    assert _pack(f, [_entry(f, 0, n), _entry(f, 1, n, g=FAKE + (64 << 20))])[0] == 0
    st, info, _ = _pack(f, [_entry(f, 0, n, group=1)])
    assert st == 0
    h, L = (f.Hyper * 8)(*[f._hyper({})] * 8), f._lib()
    opts = f.StepOpts(FAKE, 1)
    table = FAKE + 95 * GB
    for a, want in [((None, table, h, 2, 1, None, None), ARG), ((info, table, h, 1, 1, None, None), ARG),
                    ((info, table, h, 9, 1, None, None), ARG), ((info, table, None, 2, 1, None, None), ARG),
                    ((info, table, h, 2, 0, None, None), ARG), ((info, None, h, 2, 1, None, None), ARG),
                    ((info, table + 8, h, 2, 1, None, None), LAYOUT), ((info, table, h, 2, 1, table + 2, None), LAYOUT),
                    ((info, table, h, 2, 1, None, opts), ARG)]:
        i, tb, hy, nh, step, gs, o = a
        assert L.forge_multi_step(ref(i), tb, hy, nh, step, gs, ref(o), None) == want, (a, f.last_error())
    info.bytes += 4
    assert L.forge_multi_step(r(info), table, h, 2, 1, None, None, None) == ARG
    st, info, _ = _pack(f, [])
    assert L.forge_multi_step(r(info), None, None, 0, 1, None, None, None) == 0


def test_binding_refuses_host_tensors(f):
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        f.rmsnorm(x, torch.ones(128), x)
    with pytest.raises(ValueError, match="CUDA"):
        f.grouped_gemm(x, x.view(1, 4, 128), torch.zeros(1, dtype=torch.int32), x)
    with pytest.raises(ValueError, match="CUDA"):
        f.MultiStep([x], [x], opt="sgd")
    with pytest.raises(ValueError, match="scale_mode"):
        f.rmsnorm(x, x, x, scale_mode="block")
    with pytest.raises(ValueError, match="tensors"):
        f.MultiStep([x], [], opt="sgd")


def test_norm_gradient_formula_against_differences():
    g = torch.Generator().manual_seed(3)
    h, gain, dy, dh = (torch.randn(*s, dtype=R.F64, generator=g) for s in ((3, 20), (20,), (3, 20), (3, 20)))
    loss = lambda h, gain: float((R.norm(h, gain, 1e-3)[0] * dy).sum() + (h * dh).sum())  # noqa: E731
    dx, dgain = R.norm_grads(dy, h, gain, R.norm(h, gain, 1e-3)[1], dh)
    eps = 1e-5
    for grad, x, at in ((dx, h, lambda z: loss(z, gain)), (dgain, gain, lambda z: loss(h, z))):
        num = torch.empty_like(x)
        for i in range(x.numel()):
            up, down = x.clone(), x.clone()
            up.view(-1)[i] += eps
            down.view(-1)[i] -= eps
            num.view(-1)[i] = (at(up) - at(down)) / (2 * eps)
        # central differences: O(eps^2) truncation and 2^-53 |loss| / eps rounding
        assert torch.allclose(grad, num, rtol=0, atol=1e-8)


def test_multi_pack_refuses_more_chunks_than_a_grid_takes(f):
    """2^32 threads of a launch, 256 a chunk of 4096 elements: 2^36 elements are refused when they are packed."""
    from optimizer_step_weight_amd.layer import _MultiTensor
    n = 2 ** 32 - 8192

    def size(count):
        a = (_MultiTensor * count)(*[_MultiTensor(FAKE + 64 * i * GB, FAKE - 64 * GB, None, None, None, None, n, 7, f.BF16, f.BF16, 0, 0)
                                     for i in range(count)])
        return f._lib().forge_multi_table_bytes(a, count)
    assert size(16) == 16 * 72 + 16 * 4 * (2 ** 20 - 2)
    assert size(17) == -1
