"""Layer norm's gradient in rows far from 0: the lanes beyond the row's columns must not show where the
mean times the factor passes fp32, and rows in 8 bits keep to the definition."""
import pytest

torch = pytest.importorskip("torch")
sg = pytest.importorskip("spgemm_symbolic_row_amd")

import rows8_reference as rows8
import norm_reference as ref
from expert_reference import assert_within

pytestmark = pytest.mark.gpu

F32, BF, HF = torch.float32, torch.bfloat16, torch.float16


@pytest.mark.parametrize("keep", [True, "e4m3"])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("D", [4, 8, 20, 100, 136, 260, 600, 1100, 2100, 4100, 8200, 16380])
def test_large_constant_rows(D, dtype, keep):
    """Rows of c in every column, whose mean is set to c and whose factor to r = 2^9, as eps = 2^-18 makes it: n is 0 and
    dx = r (dy - mean dy)."""
    c = 2.0 ** 120   # times r: beyond fp32
    gen = torch.Generator().manual_seed(D)
    T = 5
    x = torch.randn(T, D, generator=gen)
    x[1:4] = c
    x = x.to(dtype).cuda()
    dy = torch.randn(T, D, generator=gen).to(dtype).cuda()
    w = torch.ones(D, device="cuda")
    print(f"D={D} {dtype} {keep}", flush=True)
    _, kept = sg.layer_norm(x, w, eps=2.0 ** -18, keep=keep)
    # What the forward pass kept of them, at the block's start and 256 bytes on.
    mean, rstd = kept.block[:4 * T].view(F32), kept.block[256:256 + 4 * T].view(F32)
    mean[1:4], rstd[1:4] = c, 512.0
    dx, dw, _ = sg.layer_norm_backward(dy, kept)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(dx).all()) and bool(torch.isfinite(dw).all())
    g = dy[1:4].double()
    want = 512.0 * (g - g.mean(1, keepdim=True))
    # The mean of dy: 64 additions and two roundings of 1 / D; then a subtraction, a product and the type's rounding.
    u = {F32: 2.0 ** -24, BF: 2.0 ** -8}[dtype]
    b = 512.0 * 2.0 ** -24 * (70 * g.abs().mean(1, keepdim=True) + 3 * g.abs())
    assert bool(((dx[1:4].double() - want).abs() <= b + u * (want.abs() + b)).all())


@pytest.mark.parametrize("dtype,far", [(F32, 3.0), (F32, 100.0), (BF, 10.0), (HF, 30.0)])
def test_shifted_rows_in_8_bits(dtype, far):
    """Means of `far` deviations.  The 8 bits hold x, whose rounding is 2^-4 of |x| and so a good part of a deviation
    or many: the gradients are those at the rounded rows, with the mean and the factor of x."""
    T, D = 33, 777
    gen = torch.Generator().manual_seed(7)
    x = (torch.randn(T, D, generator=gen) + far).to(dtype)
    w, b, dy = torch.randn(D, generator=gen), torch.randn(D, generator=gen), torch.randn(T, D, generator=gen).to(dtype)
    y, kept = sg.layer_norm(x.cuda(), w.cuda(), b.cuda(), keep="e4m3")
    got = sg.layer_norm_backward(dy.cuda(), kept)
    torch.cuda.synchronize()
    want = ref.layer_norm(x, w, b, 1e-5, dy, rows8.kept(x))
    assert_within(y, *want["y"], "y")
    for name, g in zip(("grad_x", "grad_weight", "grad_bias"), got):
        assert_within(g, *want[name], name)
