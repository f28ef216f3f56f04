"""ctypes declarations of the expert-layer entry points (include/spgemm.h)."""
from __future__ import annotations

import ctypes

c_i64, c_i32, c_vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p


class RouteOptions(ctypes.Structure):
    _fields_ = [("sigmoid", c_i32), ("groups", c_i32), ("top_groups", c_i32),
                ("no_renormalise", c_i32), ("scale", ctypes.c_float)]


KEPT_E4M3 = 0x45344d33  # SPGEMM_KEPT_E4M3


class ExpertsDesc(ctypes.Structure):
    _fields_ = [("tokens", c_i64), ("experts", c_i64), ("width", c_i64), ("hidden", c_i64),
                ("x_ld", c_i64), ("grad_ld", c_i64), ("k", c_i32), ("dtype", ctypes.c_int),
                ("unaligned", c_i32), ("kept_form", c_i32)]


class ExpertStepDesc(ctypes.Structure):
    _fields_ = [("tokens", c_i64), ("experts", c_i64), ("width", c_i64), ("hidden", c_i64),
                ("x_ld", c_i64), ("k", c_i32), ("dtype", ctypes.c_int),
                ("weight_dtype", ctypes.c_int), ("router_dtype", ctypes.c_int),
                ("route", RouteOptions)]


class LayerNormDesc(ctypes.Structure):
    _fields_ = [("rows", c_i64), ("width", c_i64), ("x_ld", c_i64), ("grad_ld", c_i64),
                ("dtype", ctypes.c_int), ("weight_dtype", ctypes.c_int), ("eps", ctypes.c_float),
                ("kept_form", c_i32)]


def declare(L):
    """Argument types of the expert-layer entry points."""
    st, p64 = ctypes.c_int, ctypes.POINTER(c_i64)
    L.spgemm_route.restype = st
    L.spgemm_route.argtypes = [c_i64, c_i64, c_i32, c_vp, c_i64, ctypes.c_int, c_vp, c_vp,
                               ctypes.POINTER(RouteOptions), c_vp, c_vp, c_vp]
    L.spgemm_route_backward.restype = st
    L.spgemm_route_backward.argtypes = [c_i64, c_i64, c_i32, c_vp, c_i64, ctypes.c_int, c_vp,
                                        ctypes.POINTER(RouteOptions), c_vp, c_vp, c_vp, c_vp]
    L.spgemm_dispatch_workspace.restype = c_i64
    L.spgemm_dispatch_workspace.argtypes = [c_i64, c_i32, c_i64]
    L.spgemm_dispatch.restype = st
    L.spgemm_dispatch.argtypes = [c_i64, c_i32, c_i64, c_vp, c_vp, c_vp, c_vp, c_i64, c_vp]
    L.spgemm_experts_sizes.restype = st
    L.spgemm_experts_sizes.argtypes = [ctypes.POINTER(ExpertsDesc), p64, p64, p64]
    L.spgemm_experts_forward.restype = st
    L.spgemm_experts_forward.argtypes = [ctypes.POINTER(ExpertsDesc)] + [c_vp] * 8 + [c_i64, c_vp]
    L.spgemm_experts_backward.restype = st
    L.spgemm_experts_backward.argtypes = [ctypes.POINTER(ExpertsDesc)] + [c_vp] * 10 + [c_i64, c_vp]
    L.spgemm_clip_grad_norm_workspace.restype = c_i64
    L.spgemm_clip_grad_norm_workspace.argtypes = [c_i64]
    L.spgemm_clip_grad_norm.restype = st
    L.spgemm_clip_grad_norm.argtypes = [c_i64, c_vp, c_vp, c_vp, c_vp, c_vp, ctypes.c_double,
                                        c_vp, c_vp, c_i64, c_vp]
    L.spgemm_layer_norm_sizes.restype = st
    L.spgemm_layer_norm_sizes.argtypes = [ctypes.POINTER(LayerNormDesc), p64, p64]
    L.spgemm_layer_norm_forward.restype = st
    L.spgemm_layer_norm_forward.argtypes = [ctypes.POINTER(LayerNormDesc)] + [c_vp] * 6
    L.spgemm_layer_norm_backward.restype = st
    L.spgemm_layer_norm_backward.argtypes = [ctypes.POINTER(LayerNormDesc)] + [c_vp] * 8 + [c_i64, c_vp]
    L.spgemm_expert_step_workspace.restype = st
    L.spgemm_expert_step_workspace.argtypes = [ctypes.POINTER(ExpertStepDesc), p64]
    L.spgemm_expert_step.restype = st
    L.spgemm_expert_step.argtypes = [ctypes.POINTER(ExpertStepDesc)] + [c_vp] * 12 + [c_i64, c_vp]
