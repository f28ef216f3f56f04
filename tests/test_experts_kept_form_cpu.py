"""The description's field that was reserved before rows could be kept in 8 bits: a caller that
never set it gets what it always got, through the C ABI on a machine without a GPU."""
import ctypes

import spgemm_symbolic_row_amd as sg
from spgemm_symbolic_row_amd._expert_abi import ExpertsDesc


def sizes(form):
    T, E, D, F, k = 512, 8, 256, 128, 2
    out = [ctypes.c_int64() for _ in range(3)]
    status = sg.lib().spgemm_experts_sizes(ExpertsDesc(T, E, D, F, D, D, k, 2, 0, form), *map(ctypes.byref, out))
    assert status == 0, form
    return [v.value for v in out]


def test_only_its_own_value_keeps_8_bits():
    n, F, T, D = 512 * 2, 128, 512, 256
    want = sizes(0)
    assert want[0] >= n * F * 8
    for left in (1, 2, 3, -1, 7, 0x7fffffff, -0x80000000, 0x5a5a5a5a):
        assert sizes(left) == want, left
    with open(sg.__file__.rsplit("/", 2)[0] + "/include/spgemm.h") as f:
        line = next(x for x in f if "define SPGEMM_KEPT_E4M3" in x)
    eight = sizes(int(line.split()[2], 16))
    assert T * D < eight[0] < want[0] / 2 and eight[1] == want[1]
