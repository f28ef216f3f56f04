"""Where the workspace of expert_step may begin, through the C ABI on a machine without a GPU."""
import ctypes

import spgemm_symbolic_row_amd as sg
from spgemm_symbolic_row_amd._expert_abi import ExpertStepDesc, RouteOptions


def test_a_workspace_that_atomic_operations_cannot_use_is_refused():
    L = sg.lib()
    d = ExpertStepDesc(4, 16, 64, 32, 64, 2, 2, 2, 2, RouteOptions())
    arrays = [ctypes.c_void_p(256)] * 11   # x, router, bias, active, w_in, in_scale, w_out, out_scale, y, col, val
    for at in (1, 2, 3, 257, 1026):
        assert L.spgemm_expert_step(d, *arrays, ctypes.c_void_p(at), 1 << 30, None) == -1, at
        assert b"workspace" in L.spgemm_last_error(None)
