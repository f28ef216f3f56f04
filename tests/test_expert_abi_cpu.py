"""Argument checks of the expert-layer entry points that return before any
device call, through the C ABI on a machine without a GPU."""
import ctypes

import spgemm_symbolic_row_amd as sg
from spgemm_symbolic_row_amd._expert_abi import ExpertsDesc, RouteOptions

P = ctypes.c_void_p(256)


def test_route_refuses():
    L = sg.lib()
    def route(T=4, E=16, k=2, logits=P, ld=16, dtype=0, opts=RouteOptions(), col=P, val=P):
        return L.spgemm_route(T, E, k, logits, ld, dtype, None, None, opts, col, val, None)
    assert route(T=-1) == -1 and route(E=0) == -1 and route(E=1025) == -1
    assert route(k=0) == -1 and route(k=17) == -1 and route(E=128, ld=128, k=65) == -1
    assert route(dtype=1) == -1 and route(dtype=7) == -1
    assert route(ld=15) == -1 and route(opts=None) == -1
    assert route(logits=None) == -1 and route(col=None) == -1 and route(val=None) == -1
    assert route(opts=RouteOptions(0, 3, 0, 0, 1.0)) == -1      # 3 does not divide 16
    assert route(opts=RouteOptions(0, 4, 5, 0, 1.0)) == -1
    assert route(k=5, opts=RouteOptions(0, 4, 1, 0, 1.0)) == -1  # 4 experts to pick from
    assert route(T=1 << 31) == -3
    assert b"route" in L.spgemm_last_error(None)
    assert route(T=0, logits=None, col=None, val=None) == 0
    b = L.spgemm_route_backward
    assert b(4, 16, 2, P, 16, 0, None, RouteOptions(), P, P, None, None) == -1


def test_dispatch_refuses():
    L = sg.lib()
    need = L.spgemm_dispatch_workspace(8, 2, 4)
    assert need > 0 and L.spgemm_dispatch_workspace(8, 2, 2000) == 0
    def dispatch(T=8, k=2, E=4, col=P, rp=P, ent=P, work=P, nbytes=need):
        return L.spgemm_dispatch(T, k, E, col, rp, ent, work, nbytes, None)
    assert dispatch(T=-1) == -1 and dispatch(k=0) == -1 and dispatch(E=0) == -1
    assert dispatch(col=None) == -1 and dispatch(rp=None) == -1 and dispatch(work=None) == -1
    assert dispatch(nbytes=need - 1) == -1 and dispatch(T=1 << 31) == -3


def test_experts_refuse():
    L = sg.lib()
    def desc(T=8, E=4, D=16, F=8, x_ld=16, grad_ld=16, k=2, dtype=2):
        return ExpertsDesc(T, E, D, F, x_ld, grad_ld, k, dtype, 0, 0)
    sizes = [ctypes.c_int64() for _ in range(3)]
    def size(d):
        return L.spgemm_experts_sizes(d, *map(ctypes.byref, sizes))
    assert size(desc()) == 0 and all(s.value > 0 for s in sizes)
    for bad in (dict(T=-1), dict(E=0), dict(E=1025), dict(D=0), dict(F=0), dict(x_ld=15),
                dict(k=0), dict(k=65), dict(dtype=0), dict(dtype=1)):
        assert size(desc(**bad)) == -1, bad
    assert size(desc(T=1 << 31)) == -3 and size(desc(D=1 << 25, x_ld=1 << 25)) == -3
    f = L.spgemm_experts_forward
    assert f(desc(), None, P, P, P, P, P, None, P, 1 << 40, None) == -1
    assert f(desc(), P, P, P, P, P, P, None, P, 16, None) == -1
    assert f(desc(T=0), None, None, None, None, None, None, None, None, 0, None) == 0
    b = L.spgemm_experts_backward
    assert b(desc(), P, P, P, P, None, P, P, P, P, P, 1 << 40, None) == -1
    assert b(desc(grad_ld=8), P, P, P, P, P, P, P, P, P, P, 1 << 40, None) == -1
    assert b(desc(), P, P, P, P, P, P, P, P, P, P, 16, None) == -1


def test_clip_refuses():
    L = sg.lib()
    need = L.spgemm_clip_grad_norm_workspace(1)
    ptr, size = (ctypes.c_void_p * 1)(256), (ctypes.c_int64 * 1)(4)
    def clip(n=1, g=ptr, o=ptr, s=size, t=0, m=1.0, norm=P, work=P, nbytes=need):
        ty = (ctypes.c_int32 * 1)(t)
        return L.spgemm_clip_grad_norm(n, g, o, s, ty, ty, m, norm, work, nbytes, None)
    assert clip(n=-1) == -1 and clip(g=None) == -1 and clip(norm=None) == -1
    assert clip(work=None) == -1 and clip(nbytes=need - 1) == -1
    assert clip(t=1) == -1 and clip(t=9) == -1
    assert clip(m=-1.0) == -1 and clip(m=float("nan")) == -1
    assert clip(s=(ctypes.c_int64 * 1)(-1)) == -1
    assert clip(o=(ctypes.c_void_p * 1)()) == -1


def test_sizes_that_no_launch_takes():
    """Sums over 2^35 values take 2^32 work items: refused before anything is launched."""
    L = sg.lib()
    def size(T, D):
        return L.spgemm_experts_sizes(ExpertsDesc(T, 4, D, 8, D, D, 1, 2, 0, 0), None, None, None)
    assert size((1 << 24) - 1, 2048) == 0 and size(1 << 24, 2048) == -3
    assert size((1 << 23) - 1, 4096) == 0 and size(1 << 23, 4096) == -3
    assert size(1 << 30, 8) == 0
