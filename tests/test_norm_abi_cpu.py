"""Argument checks of the layer-norm entry points that return before any device call,
through the C ABI on a machine without a GPU."""
import ctypes

import spgemm_symbolic_row_amd as sg
from spgemm_symbolic_row_amd._expert_abi import LayerNormDesc

P = ctypes.c_void_p(256)


def desc(T=8, D=16, x_ld=16, grad_ld=16, dtype=2, weight=0, eps=1e-5, form=1):
    return LayerNormDesc(T, D, x_ld, grad_ld, dtype, weight, eps, form)


def test_descriptions():
    L = sg.lib()
    kept, work = ctypes.c_int64(), ctypes.c_int64()
    def size(**k):
        return L.spgemm_layer_norm_sizes(desc(**k), ctypes.byref(kept), ctypes.byref(work))
    assert size() == 0 and kept.value >= 8 * 8 and work.value >= 2 * 16 * 4
    assert size(form=0) == 0 and kept.value == 0
    assert size(form=2) == 0 and kept.value >= 8 * (8 + 16 + 1)
    assert size(T=0) == 0
    for bad in (dict(T=-1), dict(D=0, x_ld=0, grad_ld=0), dict(D=16385, x_ld=16385, grad_ld=16385), dict(x_ld=15),
                dict(grad_ld=15), dict(dtype=1), dict(dtype=9), dict(weight=3), dict(weight=1), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(form=3), dict(form=-1)):
        assert size(**bad) == -1, bad
    assert b"layer_norm" in L.spgemm_last_error(None)
    assert size(weight=2) == 0 and size(dtype=3, weight=3) == 0
    assert size(T=1 << 31) == -3 and size(x_ld=1 << 30) == -3
    # A launch takes fewer than 2^32 work items: 64 rows to 256 of them, or 1 to 1024.
    assert size(T=(1 << 30) - 64) == 0 and size(T=1 << 30) == -3
    wide = dict(D=9000, x_ld=9000, grad_ld=9000)
    assert size(T=(1 << 22) - 1, **wide) == 0 and size(T=1 << 22, **wide) == -3
    assert L.spgemm_layer_norm_sizes(None, None, None) == -1
    assert L.spgemm_layer_norm_sizes(desc(), None, None) == 0


def test_arrays():
    L = sg.lib()
    f, b = L.spgemm_layer_norm_forward, L.spgemm_layer_norm_backward
    assert f(desc(T=0), None, None, None, None, None, None) == 0
    assert f(desc(), None, P, None, P, P, None) == -1
    assert f(desc(), P, None, None, P, P, None) == -1
    assert f(desc(), P, P, None, None, P, None) == -1
    assert f(desc(), P, P, None, P, None, None) == -1
    args = [P, P, P, P, P, P, P, P]   # x, weight, grad_y, kept, grad_x, grad_weight, grad_bias, work
    def back(form=1, nbytes=1 << 30, **none):
        return b(desc(form=form), *(None if f"a{i}" in none else a for i, a in enumerate(args)), nbytes, None)
    assert back(form=0) == -1 and back(nbytes=16) == -1
    for i in (0, 1, 2, 3, 4, 5, 7):
        assert back(**{f"a{i}": True}) == -1, i
