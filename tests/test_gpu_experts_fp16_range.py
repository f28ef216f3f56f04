"""float16 gradients keep their accuracy at any size of the incoming gradient
and of the routing weights.

The inner gradients [dg, du] and w h are held in 16 bits.  Held in units of
the size of what makes them, an element is off by 2^-11 of itself or, where it
is far smaller, by 2^-25 of the largest |w dy| of its row (for grad_x) or of
its expert (for grad_w_in), and of the expert's largest |w| (for grad_w_out).
The bounds are those of expert_reference without its absolute terms, with
twice these in their place, and the final rounding's."""
import pytest

torch = pytest.importorskip("torch")
sg = pytest.importorskip("spgemm_symbolic_row_amd")
import expert_reference as ref
from test_gpu_experts import routing, tensors

pytestmark = pytest.mark.gpu

HF = torch.float16
NAMES = ("grad_x", "grad_w_in", "grad_w_out", "grad_val")


def bounds(x, w_in, w_out, col, val, dy, monkeypatch):
    monkeypatch.setitem(ref.TINY, HF, 0.0)
    want = ref.experts(x, w_in, w_out, col, val, dy)
    monkeypatch.undo()
    extra = {n: torch.zeros_like(want[n][0]) for n in NAMES}
    top = dy.double().abs().amax(1)
    for e in range(w_in.shape[0]):
        t, i = torch.nonzero(col == e, as_tuple=True)
        if not len(t):
            continue
        w = val.double()[t, i].abs()
        row = 2.0 ** -24 * w * top[t]
        extra["grad_x"].index_add_(0, t, row[:, None] * w_in[e].double().abs().sum(0))
        extra["grad_w_in"][e] = row.max() * x.double().abs()[t].sum(0)
        extra["grad_w_out"][e] = (2.0 ** -24 * w.max() * dy.double().abs()[t].sum(0))[:, None]
    tiny = {n: 0.0 if n == "grad_val" else 2.0 ** -25 for n in NAMES}
    return {n: (want[n][0], want[n][1] + extra[n] * (1 + 2.0 ** -10) + tiny[n]) for n in NAMES}


@pytest.mark.parametrize("T,E,k,D,F", [(200, 4, 2, 64, 48), (700, 2, 2, 72, 100), (90, 40, 3, 33, 7)])
@pytest.mark.parametrize("grad,weight", [(1e-5, 0.1), (1e-4, 1e-3), (1e4, 0.5), (1.0, 1e-12),
                                         (1.0, 1e12), ("rows", 0.3)])
def test_gradients_of_any_size(T, E, k, D, F, grad, weight, monkeypatch):
    print(f"T={T} E={E} k={k} D={D} F={F} grad {grad} weight {weight}", flush=True)
    col, val = routing(T, E, k, 31, idle=0.05)
    x, w_in, w_out, dy = tensors(T, E, D, F, HF, 32)
    val = val * weight
    if grad == "rows":  # each token's gradient of its own size
        size = 10.0 ** torch.linspace(-5, 3, T)[torch.randperm(T, generator=torch.Generator().manual_seed(1))]
        dy = (dy.float() * size[:, None]).to(HF)
    else:
        dy = (dy.float() * grad).clamp(-6e4, 6e4).to(HF)
    want = bounds(x, w_in, w_out, col, val, dy, monkeypatch)
    _, kept = sg.experts(*(t.cuda() for t in (x, w_in, w_out, col, val)), keep=True)
    got = sg.experts_backward(dy.cuda(), kept)
    torch.cuda.synchronize()
    for name, g in zip(NAMES, got):
        value, bound = want[name]
        fits = value.abs() + bound < 65504 if name != "grad_val" else torch.ones_like(value, dtype=torch.bool)
        assert weight > 1 or bool(fits.any())
        ref.assert_within(g.cpu()[fits], value[fits], bound[fits], name)


def test_rows_and_weights_without_size(monkeypatch):
    """Gradients and weights that are 0, and an expert whose every row is."""
    T, E, k, D, F = 60, 3, 1, 40, 24
    col, val = routing(T, E, k, 33)
    x, w_in, w_out, dy = tensors(T, E, D, F, HF, 34)
    val[::5] = 0.0
    dy[1::5] = 0.0
    dy[(col == 2)[:, 0]] = 0.0
    want = bounds(x, w_in, w_out, col, val, dy, monkeypatch)
    _, kept = sg.experts(*(t.cuda() for t in (x, w_in, w_out, col, val)), keep=True)
    got = sg.experts_backward(dy.cuda(), kept)
    torch.cuda.synchronize()
    for name, g in zip(NAMES, got):
        ref.assert_within(g, *want[name], name)
    assert not bool(got[1][2].any()) and not bool(got[2][2].any())


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_one_token_without_a_finite_gradient(bad, monkeypatch):
    """It takes its own row and its expert's weight gradients, and nothing of other tokens and experts."""
    T, E, k, D, F = 80, 4, 1, 40, 24
    col, val = routing(T, E, k, 35)
    x, w_in, w_out, dy = tensors(T, E, D, F, HF, 36)
    dy = (dy.float() * 1e-4).to(HF)
    want = bounds(x, w_in, w_out, col, val, dy, monkeypatch)
    at = 17
    dy[at, 3] = bad
    _, kept = sg.experts(*(t.cuda() for t in (x, w_in, w_out, col, val)), keep=True)
    got = [g.cpu() for g in sg.experts_backward(dy.cuda(), kept)]
    rows = torch.arange(T) != at
    others = torch.arange(E) != int(col[at, 0])
    for name, g, keep in zip(NAMES, got, (rows, others, others, rows)):
        ref.assert_within(g[keep], want[name][0][keep], want[name][1][keep], name)
        assert not bool(torch.isfinite(g[~keep]).all())
