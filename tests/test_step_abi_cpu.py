"""Argument checks of the expert layer for a few tokens that return before any device
call, through the C ABI on a machine without a GPU."""
import ctypes

import spgemm_symbolic_row_amd as sg
from spgemm_symbolic_row_amd._expert_abi import ExpertStepDesc, RouteOptions

P = ctypes.c_void_p(256)


def desc(T=4, E=16, D=64, F=32, x_ld=64, k=2, dtype=2, weight=2, router=2, route=RouteOptions()):
    return ExpertStepDesc(T, E, D, F, x_ld, k, dtype, weight, router, route)


def test_descriptions():
    L = sg.lib()
    need = ctypes.c_int64()
    def size(**how):
        return L.spgemm_expert_step_workspace(desc(**how), ctypes.byref(need))
    assert size() == 0 and need.value >= 4 * 16 * 4 + 4 * 2 * 32 * 2
    assert size(T=0) == 0 and size(T=16) == 0
    assert size(weight=4) == 0 and size(router=0) == 0 and size(dtype=3, weight=3, router=3) == 0
    for bad in (dict(T=-1), dict(T=17), dict(E=0), dict(E=1025), dict(D=15), dict(F=15), dict(D=0), dict(F=0), dict(x_ld=63), dict(k=0),
                dict(k=17), dict(E=128, k=65), dict(dtype=0), dict(dtype=4), dict(weight=3), dict(weight=0), dict(router=3),
                dict(router=4), dict(route=RouteOptions(0, 3, 0, 0, 1.0)), dict(route=RouteOptions(0, 4, 5, 0, 1.0)),
                dict(k=5, route=RouteOptions(0, 4, 1, 0, 1.0))):
        assert size(**bad) == -1, bad
    assert size(D=(1 << 20) + 1, x_ld=1 << 23) == -3 and size(F=(1 << 20) + 1) == -3 and size(x_ld=1 << 30) == -3
    assert L.spgemm_expert_step_workspace(None, ctypes.byref(need)) == -1
    assert L.spgemm_expert_step_workspace(desc(), None) == -1


def test_arrays():
    L = sg.lib()
    def step(d=desc(), nbytes=1 << 30, none=()):
        # x, router, bias, active, w_in, in_scale, w_out, out_scale, y, col, val, work
        args = [None if i in none else P for i in range(12)]
        return L.spgemm_expert_step(d, *args, nbytes, None)
    for i in (0, 1, 4, 6, 8, 9, 10, 11):
        assert step(none=(i,)) == -1, i
    for i in (5, 7):
        assert step(desc(weight=4), none=(i,)) == -1, i
    assert step(nbytes=256) == -1
    assert step(desc(T=0), none=range(12), nbytes=0) == 0
