"""Sums over a token's entries are fp32 sums: columns of very different sizes
side by side, and entries that cancel, each against a bound of its own."""
import pytest

torch = pytest.importorskip("torch")
sg = pytest.importorskip("spgemm_symbolic_row_amd")
import expert_reference as ref
from test_gpu_experts import routing, tensors

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("T,E,k,D,F", [(70, 3, 2, 200, 64), (900, 2, 2, 136, 40)])
def test_columns_of_very_different_sizes(T, E, k, D, F):
    """Column d of y takes the size of row d of W_out, column d of dx that of column d of W_in:
    every column is held to its own size, whatever its neighbours hold."""
    print(f"columns T={T} E={E} k={k} D={D} F={F}", flush=True)
    col, val = routing(T, E, k, 21)
    x, w_in, w_out, dy = tensors(T, E, D, F, BF, 22)
    small = 2.0 ** -(torch.arange(D) * 37 % 61).float()
    small[:8] = 2.0 ** 20   # what a padded column could be mistaken for
    x[:, :8] = x[:, :8] * 2.0 ** -20
    w_in, w_out = (w_in * small).to(BF), (w_out * small[:, None]).to(BF)
    dy = (dy / small.clamp(min=2.0 ** -30)).to(BF)
    want = ref.experts(x, w_in, w_out, col, val, dy)
    y, kept = sg.experts(*(t.cuda() for t in (x, w_in, w_out, col, val)), keep=True)
    got = sg.experts_backward(dy.cuda(), kept)
    torch.cuda.synchronize()
    ref.assert_within(y, *want["y"], "y")
    for name, g in zip(("grad_x", "grad_w_in", "grad_w_out", "grad_val"), got):
        ref.assert_within(g, *want[name], name)


def test_entries_that_cancel():
    """Two experts whose W_out differ in one place of F, with weights 1 and -1.  Their hidden
    vectors are the same, so the rounding of h enters through the difference alone."""
    T, D, F = 300, 72, 8
    x, w_in, w_out, _ = tensors(T, 2, D, F, BF, 23)
    w_in[1] = w_in[0]
    w_out[1] = w_out[0]
    w_out[1, :, 3] *= 1.0 + 2.0 ** -6
    col = torch.tensor([[0, 1]], dtype=torch.int32).repeat(T, 1)
    val = torch.tensor([[1.0, -1.0]]).repeat(T, 1)
    y, _ = sg.experts(*(t.cuda() for t in (x, w_in, w_out, col, val)), keep=True)
    torch.cuda.synchronize()
    p = x.double() @ w_in[0].double().T
    mag = x.double().abs() @ w_in[0].double().abs().T
    g, u = p[:, :F], p[:, F:]
    h = torch.nn.functional.silu(g) * u
    dG, dU = 2 * D * ref.EPS * mag[:, :F], 2 * D * ref.EPS * mag[:, F:]
    dh = 1.1 * dG * u.abs() + (g.abs() + 1.1 * dG) * dU + 3 * ref.FUN * h.abs()
    dh = dh + ref.U[BF] * (h.abs() + dh)
    a, b = w_out[0].double(), w_out[1].double()
    want = h @ (a - b).T
    bound = dh @ (a - b).abs().T + 2 * (F + 2) * ref.EPS * (h.abs() + dh) @ (a.abs() + b.abs()).T
    ref.assert_within(y, want, bound + ref.U[BF] * (want.abs() + bound), "y")
