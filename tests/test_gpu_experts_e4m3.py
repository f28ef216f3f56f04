"""The expert layer's gradients from an input kept in 8 bits: those at the values that
the 8 bits stand for, to the last bit."""
import pytest

torch = pytest.importorskip("torch")
sg = pytest.importorskip("spgemm_symbolic_row_amd")
import expert_reference as ref
import rows8_reference as rows8
from test_gpu_experts import routing, tensors

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
NAMES = ("grad_x", "grad_w_in", "grad_w_out", "grad_val")


def bits(t):
    return t.view(torch.int32 if t.dtype == torch.float32 else torch.int16)


CASES = [
    # T, E, k, D, F, type, routing
    (1, 4, 1, 8, 8, BF, {}),
    (1, 8, 8, 64, 72, HF, {}),
    (3, 5, 2, 33, 7, BF, {}),
    (17, 3, 3, 100, 36, HF, dict(gaps=True)),
    (130, 2, 1, 129, 200, BF, {}),
    (129, 7, 2, 264, 88, HF, dict(hot=0.9)),
    (300, 64, 1, 72, 40, BF, {}),
    (600, 2, 2, 520, 136, HF, dict(idle=0.1)),
    (50, 6, 2, 1, 1, BF, {}),
    (40, 3, 2, 2056, 136, BF, {}),
    (1500, 4, 2, 136, 72, BF, dict(idle=0.02, hot=0.3)),
]


@pytest.mark.parametrize("T,E,k,D,F,dtype,how", CASES)
def test_gradients(T, E, k, D, F, dtype, how):
    print(f"experts T={T} E={E} k={k} D={D} F={F} {dtype} {how}", flush=True)
    col, val = routing(T, E, k, T + E, **how)
    x, w_in, w_out, dy = tensors(T, E, D, F, dtype, D)
    at = rows8.kept(x).to(dtype)
    want = ref.experts(at, w_in, w_out, col, torch.where(col < 0, 0.0, val), dy)
    x, at, w_in, w_out, col, val, dy = (t.cuda() for t in (x, at, w_in, w_out, col, val, dy))
    y, kept = sg.experts(x, w_in, w_out, col, val, keep="e4m3")
    y2, kept_x = sg.experts(x, w_in, w_out, col, val, keep=True)
    assert torch.equal(y, y2)
    x.fill_(float("nan"))   # it need not stay
    got = sg.experts_backward(dy, kept)
    again = sg.experts_backward(dy, kept)
    _, kept_x = sg.experts(at, w_in, w_out, col, val, keep=True)
    same = sg.experts_backward(dy, kept_x)
    torch.cuda.synchronize()
    for name, g, h, s in zip(NAMES, got, again, same):
        ref.assert_within(g, *want[name], name)
        assert torch.equal(bits(g), bits(h)), f"{name} differs between two calls"
        assert torch.equal(bits(g), bits(s)), f"{name} differs from the gradient at the kept values"


def test_strided_rows():
    T, E, k, D, F = 37, 5, 2, 200, 48
    col, val = routing(T, E, k, 1)
    x, w_in, w_out, dy = tensors(T, E, D, F, BF, 2)
    col, val, w_in, w_out, dy = (t.cuda() for t in (col, val, w_in, w_out, dy))
    want = sg.experts_backward(dy, sg.experts(x.cuda(), w_in, w_out, col, val, keep="e4m3")[1])
    for ld, off in ((D + 8, 0), (D + 3, 0), (D, 1), (D + 8, 5)):
        buf = torch.full((T * ld + off + 8,), float("nan"), dtype=BF, device="cuda")
        v = buf[off:off + T * ld].view(T, ld)[:, :D]
        v.copy_(x)
        _, kept = sg.experts(v, w_in, w_out, col, val, keep="e4m3")
        g = buf.new_full((T * ld + off + 8,), float("nan"))[off:off + T * ld].view(T, ld)[:, :D]
        g.copy_(dy)
        assert all(torch.equal(p, q) for p, q in zip(want, sg.experts_backward(g, kept)))


def test_what_is_kept_is_small():
    T, E, k, D, F = 4096, 8, 4, 512, 256
    col, val = routing(T, E, k, 3)
    x, w_in, w_out, _ = (t.cuda() for t in tensors(T, E, D, F, BF, 4))
    _, kept = sg.experts(x, w_in, w_out, col.cuda(), val.cuda(), keep="e4m3")
    # The rows and their scales, and 16 bytes an entry and 8 a tile of the dispatch.
    assert kept.x is None and kept.block.numel() < T * (D + D // 128 + 32 * k) + 20000
    assert sg.experts(x, w_in, w_out, col.cuda(), val.cuda(), keep=True)[1].block.numel() > T * k * 8 * F


def test_rows_that_are_not_finite_stay_alone():
    """Tokens of other experts have the gradients that they had."""
    T, E, D, F = 64, 4, 136, 40
    for dtype in (BF, HF):
        x, w_in, w_out, dy = (t.cuda() for t in tensors(T, E, D, F, dtype, 6))
        col = (torch.arange(T, dtype=torch.int32, device="cuda") % E)[:, None].contiguous()
        val = torch.ones(T, 1, device="cuda")
        want = sg.experts_backward(dy, sg.experts(x, w_in, w_out, col, val, keep="e4m3")[1])
        x[1, 130], x[5, 0] = float("inf"), float("nan")   # both of expert 1
        got = sg.experts_backward(dy, sg.experts(x, w_in, w_out, col, val, keep="e4m3")[1])
        rows = col[:, 0] != 1
        assert torch.equal(got[0][rows], want[0][rows]) and torch.equal(got[3][rows], want[3][rows])
        assert bool(torch.isnan(got[0][1]).all()) and bool(torch.isnan(got[0][5]).all())
        for g, w in zip(got[1:3], want[1:3]):
            assert torch.equal(g[[0, 2, 3]], w[[0, 2, 3]]) and bool(torch.isnan(g[1]).any())


def test_graph_replays_and_streams():
    T, E, k, D, F = 300, 6, 2, 264, 72
    x, w_in, w_out, dy = (t.cuda() for t in tensors(T, E, D, F, BF, 8))
    col, val = (t.cuda() for t in routing(T, E, k, 9))
    def step():
        y, kept = sg.experts(x, w_in, w_out, col, val, keep="e4m3")
        return (y, *sg.experts_backward(dy, kept))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for i in range(4):
        x.copy_(torch.randn(T, D, device="cuda"))
        dy.copy_(torch.randn(T, D, device="cuda"))
        c, v = routing(T, E, k, 20 + i, idle=0.2)
        col.copy_(c)
        val.copy_(v)
        g.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, step())), i
    # The block that a pass on one stream left is read on another.
    want = step()[1:]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        _, kept = sg.experts(x, w_in, w_out, col, val, keep="e4m3")
    side.synchronize()
    at, size = kept.block.data_ptr(), kept.block.numel()
    torch.cuda._sleep(400_000_000)
    got = sg.experts_backward(dy, kept)
    del kept
    with torch.cuda.stream(side):
        new = torch.empty(size, dtype=torch.uint8, device="cuda")
    busy = not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert busy and new.data_ptr() != at
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_no_tokens_and_refusals():
    E, D, F = 3, 16, 8
    w_in = torch.randn(E, 2 * F, D, device="cuda").to(BF)
    w_out = torch.randn(E, D, F, device="cuda").to(BF)
    x = torch.empty(0, D, device="cuda", dtype=BF)
    col, val = torch.empty(0, 2, device="cuda", dtype=torch.int32), torch.empty(0, 2, device="cuda")
    y, kept = sg.experts(x, w_in, w_out, col, val, keep="e4m3")
    got = sg.experts_backward(x, kept)
    assert y.shape == got[0].shape == (0, D) and got[3].shape == (0, 2)
    assert torch.count_nonzero(got[1]) == 0 and torch.count_nonzero(got[2]) == 0
    for keep in ("8bit", "", "E4M3"):
        with pytest.raises(ValueError):
            sg.experts(x, w_in, w_out, col, val, keep=keep)
    x = torch.randn(4, D, device="cuda").to(BF)
    col, val = (t.cuda() for t in routing(4, E, 2, 0))
    _, kept = sg.experts(x, w_in, w_out, col, val, keep="e4m3")
    for error, g in ((ValueError, x[:3]), (TypeError, x.half()), (TypeError, x.cpu()),
                     (TypeError, x.clone().requires_grad_())):
        with pytest.raises(error):
            sg.experts_backward(g, kept)
