"""Structures and argument types of include/forge_layer.h.  Without torch: the library's host calls need none."""
from __future__ import annotations

import ctypes

from . import Hyper, StepOpts, Tensor


class _MultiTensor(ctypes.Structure):
    _fields_ = [("W", ctypes.c_void_p), ("g", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("seed", ctypes.c_uint64), ("w_dtype", ctypes.c_int32), ("g_dtype", ctypes.c_int32),
                ("group", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class _MultiInfo(ctypes.Structure):
    _fields_ = [("bytes", ctypes.c_int64), ("chunks", ctypes.c_int64), ("tensors", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("opt", ctypes.c_int32), ("m_dtype", ctypes.c_int32),
                ("v_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def declare(L) -> None:
    """Argument types of the entry points (called once, when the library is loaded)."""
    P = ctypes.POINTER
    T, H, O = P(Tensor), P(Hyper), P(StepOpts)
    st, i32, i64, u64, f32, vp = (ctypes.c_int, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_float,
                                  ctypes.c_void_p)
    L.forge_rmsnorm.argtypes = [T, T, T, f32, T, T, i32, vp, vp, vp]
    L.forge_rmsnorm_backward.argtypes = [T, T, T, T, vp, T, T, vp, i64, vp]
    L.forge_rmsnorm_backward_workspace_bytes.argtypes = [i64, i64]
    L.forge_grouped_gemm.argtypes = [T, T, vp, i32, T, vp]
    L.forge_grouped_dgrad.argtypes = [T, T, vp, i32, T, vp]
    L.forge_grouped_wgrad.argtypes = [T, T, vp, i32, T, vp]
    L.forge_grouped_wgrad_step.argtypes = [T, T, vp, i32, T, T, T, H, i32, i64, u64, O, vp]
    L.forge_multi_table_bytes.argtypes = [P(_MultiTensor), i32]
    L.forge_multi_pack.argtypes = [P(_MultiTensor), i32, i32, i32, i32, vp, i64, P(_MultiInfo)]
    L.forge_multi_step.argtypes = [P(_MultiInfo), vp, H, i32, i64, vp, O, vp]
    for f in ("forge_rmsnorm", "forge_rmsnorm_backward", "forge_grouped_gemm", "forge_grouped_dgrad",
              "forge_grouped_wgrad", "forge_grouped_wgrad_step", "forge_multi_pack", "forge_multi_step"):
        getattr(L, f).restype = st
    for f in ("forge_rmsnorm_backward_workspace_bytes", "forge_multi_table_bytes"):
        getattr(L, f).restype = i64
