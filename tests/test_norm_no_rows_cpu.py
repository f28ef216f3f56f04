"""Layer norm's gradient without rows: which arrays may be missing, through the C ABI on a
machine without a GPU."""
import ctypes

import spgemm_symbolic_row_amd as sg
from spgemm_symbolic_row_amd._expert_abi import LayerNormDesc

P = ctypes.c_void_p(256)


def test_the_weight_is_read_without_rows_too():
    """So a missing one is refused before anything is launched."""
    for dtype, weight, form in ((0, 0, 1), (2, 0, 1), (3, 3, 2)):
        for width in (1, 16, 600, 16384):
            d = LayerNormDesc(0, width, width, width, dtype, weight, 1e-5, form)
            # x, weight, grad_y, kept, grad_x, grad_weight, grad_bias, work
            status = sg.lib().spgemm_layer_norm_backward(d, None, None, None, None, None, P, P, P, 1 << 30, None)
            assert status == -1
            assert b"null array" in sg.lib().spgemm_last_error(None)
