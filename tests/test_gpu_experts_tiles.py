"""Every form of the products over several slices of K with data, full ones and a
last one that ends inside, and weight gradients with more tiles than work groups."""
import pytest

torch = pytest.importorskip("torch")
sg = pytest.importorskip("spgemm_symbolic_row_amd")
import expert_reference as ref
from test_gpu_experts import routing, tensors

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
NAMES = ("grad_x", "grad_w_in", "grad_w_out", "grad_val")


def check(T, E, k, D, F, dtype, make=lambda t: t.cuda(), **how):
    print(f"T={T} E={E} k={k} D={D} F={F} {dtype} {how}", flush=True)
    col, val = routing(T, E, k, T + D, **how)
    x, w_in, w_out, dy = tensors(T, E, D, F, dtype, F)
    want = ref.experts(x, w_in, w_out, col, val, dy)
    y, kept = sg.experts(make(x), w_in.cuda(), w_out.cuda(), col.cuda(), val.cuda(), keep=True)
    got = sg.experts_backward(make(dy), kept)
    torch.cuda.synchronize()
    ref.assert_within(y, *want["y"], "y")
    for name, g in zip(NAMES, got):
        ref.assert_within(g, *want[name], name)


@pytest.mark.parametrize("T,E,k,D,F,dtype,how", [
    # 128 x 256 tiles of 6 to 16 slices; 288 tiles of W_in's gradient, some 220 tokens to an expert
    (1777, 24, 3, 1000, 344, BF, {}),
    (1777, 24, 3, 1000, 344, HF, {}),
    # 128 x 128 tiles
    (300, 3, 2, 328, 200, BF, {}),
    # 256 x 256 tiles, several of an expert
    (1100, 4, 2, 328, 200, HF, dict(hot=0.3)),
    # both weight gradients with more tiles than work groups, uneven experts
    (3100, 30, 2, 776, 520, BF, dict(hot=0.4)),
])
def test_several_slices(T, E, k, D, F, dtype, how):
    check(T, E, k, D, F, dtype, **how)


def test_more_tiles_than_work_groups_with_empty_experts():
    """Half the experts have no token."""
    T, E, k, D, F = 2100, 36, 1, 776, 264
    col, val = routing(T, E // 2, k, 41)
    col = col * 2
    x, w_in, w_out, dy = tensors(T, E, D, F, BF, 42)
    want = ref.experts(x, w_in, w_out, col, val, dy)
    _, kept = sg.experts(*(t.cuda() for t in (x, w_in, w_out, col, val)), keep=True)
    got = sg.experts_backward(dy.cuda(), kept)
    torch.cuda.synchronize()
    for name, g in zip(NAMES, got):
        ref.assert_within(g, *want[name], name)
    assert not bool(got[1][1::2].any()) and not bool(got[2][1::2].any())


@pytest.mark.parametrize("T,E,k", [(600, 2, 2), (520, 8, 1), (520, 200, 2)])
def test_far_rows_of_several_slices(T, E, k):
    """Rows over more than 4 GB, so that the products' pointers advance slice by slice; tiles of
    256 x 256, 128 x 128 and 128 x 256.  x and the gradient of y lie in columns of their own."""
    D, F, ld = 328, 24, 1 << 22
    buf = torch.empty(T * ld, dtype=BF, device="cuda").view(T, ld)
    free = [0, 336]
    def far(t):
        at = free.pop(0)
        v = buf[:, at:at + D]
        v.copy_(t.cuda())
        return v
    check(T, E, k, D, F, BF, make=far)
