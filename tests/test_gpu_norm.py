"""Layer norm, its gradient and rows kept in 8 bits, against a plain 64-bit form, with
error bounds derived in norm_reference."""
import pytest

torch = pytest.importorskip("torch")
sg = pytest.importorskip("spgemm_symbolic_row_amd")
import norm_reference as ref
import rows8_reference as rows8
from expert_reference import assert_within

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
NAMES = ("grad_x", "grad_weight", "grad_bias")


def tensors(T, D, dtype, wtype, seed, spread=1.0, shift=0.0):
    gen = torch.Generator().manual_seed(seed)
    def r(*s):
        return torch.randn(*s, generator=gen)
    x = (r(T, D) * spread * (1 + r(T, 1).abs()) + shift).to(dtype)
    return x, (1 + 0.3 * r(D)).to(wtype), (0.2 * r(D)).to(wtype), r(T, D).to(dtype)


def check(x, w, b, dy, eps=1e-5, keep=True, dev=None):
    """One forward and two backward passes against the reference; dev: the tensors as given to the calls."""
    want = ref.layer_norm(x, w, b, eps, dy, rows8.kept(x) if keep == "e4m3" else None)
    gx, gw, gb, gdy = dev or [None if t is None else t.cuda() for t in (x, w, b, dy)]
    plain = sg.layer_norm(gx, gw, gb, eps)
    y, kept = sg.layer_norm(gx, gw, gb, eps, keep=keep)
    got = sg.layer_norm_backward(gdy, kept)
    again = sg.layer_norm_backward(gdy, kept)
    torch.cuda.synchronize()
    assert torch.equal(plain, y)
    assert y.is_contiguous() and y.dtype == x.dtype
    assert_within(y, *want["y"], "y")
    assert (got[2] is None) == (b is None)
    for name, g, h in zip(NAMES, got, again):
        if g is not None:
            assert g.dtype == (x.dtype if name == "grad_x" else w.dtype)
            assert_within(g, *want[name], name)
            assert torch.equal(g, h), f"{name} differs between two calls"
    return y, got


WIDTHS = [1, 2, 7, 8, 100, 127, 128, 129, 250, 511, 512, 513, 1000, 1001, 1024, 1032, 2047, 2048, 2049,
          4096, 4100, 8192, 8200, 16383, 16384]


@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("D", WIDTHS)
def test_widths(D, dtype):
    T = 37 if D < 2000 else 9
    print(f"T={T} D={D} {dtype}", flush=True)
    for keep in (True, "e4m3"):
        for wtype in {F32, dtype}:
            x, w, b, dy = tensors(T, D, dtype, wtype, D)
            check(x, w, b if D % 2 else None, dy, keep=keep)


@pytest.mark.parametrize("T,D,dtype", [(1, 64, BF), (1, 2048, F32), (2, 300, HF), (63, 128, BF), (64, 128, F32),
                                       (65, 100, HF), (1025, 40, BF), (40000, 24, BF), (5000, 130, F32),
                                       (3001, 1001, HF), (2100, 2048, BF), (1500, 4096, HF), (700, 8192, BF),
                                       (600, 10000, F32)])
def test_rows(T, D, dtype):
    """More rows than one turn of the gradient's work groups, and fewer than one work group's."""
    print(f"T={T} D={D} {dtype}", flush=True)
    for keep in (True, "e4m3"):
        check(*tensors(T, D, dtype, F32, T), keep=keep)


@pytest.mark.parametrize("dtype", [F32, BF, HF])
def test_strides_and_alignment(dtype):
    T, D = 21, 200
    x, w, b, dy = tensors(T, D, dtype, dtype, 5)
    for ld, off in ((D + 8, 0), (D + 3, 0), (D, 1), (D + 7, 5)):
        def strided(t):
            buf = torch.full((T * ld + off + 8,), float("nan"), dtype=dtype, device="cuda")
            v = buf[off:off + T * ld].view(T, ld)[:, :D]
            v.copy_(t)
            return v
        def shifted(t):
            buf = torch.full((D + off,), float("nan"), dtype=dtype, device="cuda")
            buf[off:].copy_(t)
            return buf[off:]
        for keep in (True, "e4m3"):
            check(x, w, b, dy, keep=keep, dev=(strided(x), shifted(w), shifted(b), strided(dy)))


def test_large_means_zeros_and_eps():
    for dtype, shift in ((F32, 300.0), (BF, 50.0), (HF, -400.0)):
        check(*tensors(33, 777, dtype, F32, 7, shift=shift))
    x, w, b, dy = tensors(9, 260, F32, F32, 8)
    x[3] = 0.0
    x[4] = 2.0
    x[5] *= 1e-12
    for keep in (True, "e4m3"):
        check(x, w, b, dy, eps=1e-3, keep=keep)
        check(x[6:], w, b, dy[6:], eps=0.0, keep=keep)
    check(x * 1e15, w, b, dy, eps=1.0)   # squares up to 1e31


def test_rows_without_finite_values_stay_alone():
    """A row that holds an infinity or a NaN leaves the other rows' y and dx as they are, kept in 8 bits or not."""
    for dtype in (F32, BF, HF):
        x, w, b, dy = (t.cuda() for t in tensors(40, 300, dtype, F32, 9))
        for keep in (True, "e4m3"):
            y, kept = sg.layer_norm(x, w, b, keep=keep)
            dx = sg.layer_norm_backward(dy, kept)[0]
            bad = x.clone()
            bad[7, 290], bad[8, 3], bad[30] = float("inf"), float("nan"), float("-inf")
            y2, kept = sg.layer_norm(bad, w, b, keep=keep)
            dx2, dw2, _ = sg.layer_norm_backward(dy, kept)
            rows = torch.tensor([i for i in range(40) if i not in (7, 8, 30)], device="cuda")
            assert torch.equal(y[rows], y2[rows]) and torch.equal(dx[rows], dx2[rows])
            for r in (7, 8, 30):
                assert bool(torch.isnan(y2[r]).any()) and bool(torch.isnan(dx2[r]).all())
            assert bool(torch.isnan(dw2).all())


@pytest.mark.parametrize("dtype", [F32, BF, HF])
def test_codes_over_the_whole_range(dtype):
    """Rows of every size that the type has, its largest and subnormal values, ties between two codes.  The codes are
    looked at through the gradient of the weight: with one row, dw = dy (x - m) r."""
    gen = torch.Generator().manual_seed(3)
    top = torch.finfo(dtype).max
    rows = [torch.randn(400, generator=gen).double() * 2.0 ** e for e in (-140, -126, -118, -100, -24, -16, -9, 0, 9, 15)]
    rows = [r.clamp(-top, top).to(dtype) for r in rows]
    ties = torch.tensor([448.0, 1.0625, 1.1875, 17.0, 18.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11, 440.0, -432.0,
                         -416.0, 0.0, -0.0] * 20)
    rows += [ties.to(dtype), (ties * 1.25).to(dtype), torch.full((130,), top, dtype=dtype) * torch.linspace(-1, 1, 130).to(dtype)]
    for i, row in enumerate(rows):
        x = row[None]
        want = rows8.kept(x)
        D = x.shape[1]
        one = torch.ones(D, device="cuda")
        _, kept = sg.layer_norm(x.cuda(), one, keep="e4m3")
        _, kept_x = sg.layer_norm(want.to(dtype).cuda(), one, keep=True)
        assert torch.equal(want.to(dtype).double(), want), "what is kept is exact in the type"
        # A mean of 0 and a factor of 1 beside both (a block begins with them, at multiples of 256 bytes): then dw is
        # dy x.
        for k in (kept, kept_x):
            k.block[:4].view(F32).fill_(0.0)
            k.block[256:260].view(F32).fill_(1.0)
        dy = torch.randn(1, D, generator=gen).to(dtype).cuda()
        a, b = sg.layer_norm_backward(dy, kept), sg.layer_norm_backward(dy, kept_x)
        torch.cuda.synchronize()
        for p, q in zip(a[:2], b[:2]):
            assert torch.equal(p.view(torch.int32 if p.dtype == F32 else torch.int16),
                               q.view(torch.int32 if q.dtype == F32 else torch.int16)), i


def test_gradients_against_differences():
    """The formula's gradient beside central differences of the forward pass."""
    T, D = 3, 40
    x, w, b, dy = tensors(T, D, F32, F32, 11)
    _, kept = sg.layer_norm(x.cuda(), w.cuda(), b.cuda(), keep=True)
    got = [g.double().cpu() for g in sg.layer_norm_backward(dy.cuda(), kept)]
    def loss(x, w, b):
        return (ref.layer_norm(x, w, b, 1e-5)["y"][0] * dy.double()).sum()
    base = [t.double() for t in (x, w, b)]
    for which, g in enumerate(got):
        for i in range(0, base[which].numel(), 7):
            h, ends = 1e-5, []
            for sign in (1, -1):
                args = [t.clone() for t in base]
                args[which].view(-1)[i] += sign * h
                ends.append(loss64(*args, dy))
            # Differences: h^2 of the third derivative, and 2^-52 of the loss over h.
            assert abs((ends[0] - ends[1]) / (2 * h) - g.view(-1)[i]) < 2e-5 * (1 + g.abs().max())


def loss64(x, w, b, dy):
    m = x.mean(1, keepdim=True)
    v = ((x - m) ** 2).mean(1, keepdim=True)
    return float((((x - m) / torch.sqrt(v + 1e-5) * w + b) * dy.double()).sum())


def test_no_rows():
    w = torch.ones(30, device="cuda", dtype=BF)
    x = torch.empty(0, 30, device="cuda", dtype=BF)
    for keep in (True, "e4m3"):
        y, kept = sg.layer_norm(x, w, w, keep=keep)
        dx, dw, db = sg.layer_norm_backward(x, kept)
        assert y.shape == dx.shape == (0, 30)
        assert torch.count_nonzero(dw) == 0 and torch.count_nonzero(db) == 0


def test_eight_bits_need_no_x():
    """After the forward pass x may change."""
    x, w, b, dy = (t.cuda() for t in tensors(50, 600, BF, BF, 13))
    _, kept = sg.layer_norm(x, w, b, keep="e4m3")
    want = sg.layer_norm_backward(dy, kept)
    x.fill_(float("nan"))
    for p, q in zip(want, sg.layer_norm_backward(dy, kept)):
        assert torch.equal(p, q)
    assert kept.block.numel() < 50 * 600 * 1.2


def test_graph_replays():
    """Forward and backward in one captured graph, replayed over changed inputs with eager work between."""
    for keep in (True, "e4m3"):
        x, w, b, dy = (t.cuda() for t in tensors(300, 1000, BF, F32, 17))
        def step():
            y, kept = sg.layer_norm(x, w, b, keep=keep)
            return (y, *sg.layer_norm_backward(dy, kept))
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        for i in range(4):
            x.copy_(torch.randn_like(x, dtype=F32))
            dy.copy_(torch.randn_like(x, dtype=F32))
            g.replay()
            got = [t.clone() for t in out]
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, step())), i


def test_backward_on_another_stream():
    x, w, b, dy = (t.cuda() for t in tensors(512, 2048, BF, BF, 19))
    want = [t.clone() for t in sg.layer_norm_backward(dy, sg.layer_norm(x, w, b, keep="e4m3")[1])]
    torch.cuda.synchronize()
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    with torch.cuda.stream(side):
        _, kept = sg.layer_norm(x, w, b, keep="e4m3")
    side.synchronize()
    at, size = kept.block.data_ptr(), kept.block.numel()
    torch.cuda._sleep(400_000_000)
    got = sg.layer_norm_backward(dy, kept)
    del kept
    with torch.cuda.stream(side):
        new = torch.empty(size, dtype=torch.uint8, device="cuda")
    busy = not main.query()
    main.synchronize()
    assert busy and new.data_ptr() != at
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_refusals():
    x, w, b, dy = (t.cuda() for t in tensors(4, 16, BF, F32, 23))
    def bad(error, *a, **k):
        with pytest.raises(error):
            sg.layer_norm(*a, **k)
    bad(ValueError, x[0], w)
    bad(TypeError, x.t(), torch.ones(4, device="cuda"))
    bad(TypeError, x.int(), w)
    bad(TypeError, x.double(), w)
    bad(TypeError, x, w.half())
    bad(TypeError, x, w, b.bfloat16())
    bad(ValueError, x, w[:15])
    bad(ValueError, x, w, b[:, None])
    bad(TypeError, x, w.cpu())
    bad(TypeError, x, torch.ones(32, device="cuda")[::2])
    bad(ValueError, x, w, keep="8bit")
    bad(ValueError, x, w, keep=2)
    bad(sg.SpgemmError, x, w, eps=-1.0)
    bad(sg.SpgemmError, x, w, eps=float("nan"))
    bad(sg.SpgemmError, torch.zeros(1, 16385, device="cuda"), torch.ones(16385, device="cuda"))
    bad(TypeError, x, w.clone().requires_grad_())
    bad(TypeError, x[:1].expand(4, 16), w)
    _, kept = sg.layer_norm(x, w, keep=True)
    for error, g in ((ValueError, dy[:3]), (TypeError, dy.float()), (TypeError, dy.cpu()),
                     (TypeError, dy.t().contiguous().t()), (TypeError, dy.clone().requires_grad_())):
        with pytest.raises(error):
            sg.layer_norm_backward(g, kept)
