"""The experts' products, their gradients and the dispatch, against a plain
64-bit form, with error bounds derived in expert_reference."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
sg = pytest.importorskip("spgemm_symbolic_row_amd")
import expert_reference as ref

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def routing(T, E, k, seed, idle=0.0, hot=0.0, gaps=False):
    """Distinct experts per row, rising; `hot`: rows that all pick experts 0..k-1."""
    rng = np.random.default_rng(seed)
    col = np.full((T, k), -1, np.int32)
    for t in range(T):
        if rng.random() < idle:
            continue
        m = int(rng.integers(0, k + 1)) if gaps else k
        c = np.arange(k) if rng.random() < hot else rng.choice(E, size=k, replace=False)
        col[t, :m] = np.sort(c[:m])
    val = rng.normal(size=(T, k)).astype(np.float32)
    val[col < 0] = np.nan if gaps else 0.0   # empty slots are not read
    return torch.from_numpy(col), torch.from_numpy(val)


def tensors(T, E, D, F, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    def r(*s, scale=1.0):
        return (torch.randn(*s, generator=gen) * scale).to(dtype)
    return r(T, D), r(E, 2 * F, D, scale=D ** -0.5), r(E, D, F, scale=F ** -0.5), r(T, D)


CASES = [
    # T, E, k, D, F, type, routing
    (1, 4, 1, 8, 8, BF, {}),
    (1, 8, 8, 64, 72, HF, {}),
    (3, 5, 2, 33, 7, BF, {}),                     # no row begins at 16 bytes
    (17, 3, 3, 100, 36, HF, dict(gaps=True)),
    (40, 16, 4, 256, 128, BF, dict(idle=0.3)),
    (130, 2, 1, 64, 200, BF, {}),
    (129, 7, 2, 264, 88, HF, dict(hot=0.9)),      # experts of very different loads
    (300, 64, 1, 72, 40, BF, {}),                 # experts without tokens
    (600, 2, 2, 520, 136, BF, dict(idle=0.1)),    # several row tiles of one expert
    (513, 1, 1, 128, 264, HF, {}),
    (50, 6, 2, 1, 1, BF, {}),
    (200, 1024, 3, 16, 24, BF, {}),
    (33, 4, 2, 127, 65, HF, dict(gaps=True)),
    (4, 64, 6, 264, 136, BF, {}),                 # few entries: each on its own
    (7, 80, 5, 71, 50, HF, dict(gaps=True)),
    (1, 3, 2, 2056, 520, BF, {}),
    (60, 40, 2, 520, 104, BF, dict(hot=0.9)),     # few rows to most experts, several tiles of one
    (31, 32, 4, 40, 2064, HF, dict(idle=0.2)),
]


@pytest.mark.parametrize("T,E,k,D,F,dtype,how", CASES)
def test_experts_and_gradients(T, E, k, D, F, dtype, how):
    print(f"experts T={T} E={E} k={k} D={D} F={F} {dtype} {how}", flush=True)
    col, val = routing(T, E, k, T + E, **how)
    x, w_in, w_out, dy = tensors(T, E, D, F, dtype, D)
    want = ref.experts(x, w_in, w_out, col, torch.where(col < 0, 0.0, val), dy)
    dev = [t.cuda() for t in (x, w_in, w_out, col, val)]
    y = sg.experts(*dev)
    y2, kept = sg.experts(*dev, keep=True)
    got = sg.experts_backward(dy.cuda(), kept)
    again = sg.experts_backward(dy.cuda(), kept)
    torch.cuda.synchronize()
    ref.assert_within(y, *want["y"], "y")
    ref.assert_within(y2, *want["y"], "y, kept")
    for name, g, h in zip(("grad_x", "grad_w_in", "grad_w_out", "grad_val"), got, again):
        ref.assert_within(g, *want[name], name)
        assert torch.equal(g, h), f"{name} differs between two calls"
    empty = col < 0
    assert bool((got[3].cpu()[empty] == 0).all())
    none = empty.all(1)
    assert bool((y.cpu()[none] == 0).all()) and bool((got[0].cpu()[none] == 0).all())


def test_many_tokens_of_few_experts():
    """Rows of 256 to a tile, and K longer than one weight gradient's slice."""
    test_experts_and_gradients(1500, 4, 2, 136, 72, BF, dict(idle=0.02, hot=0.3))


@pytest.mark.parametrize("T,E,D,F", [(4500, 1, 40, 24), (4600, 9, 1032, 264)])
def test_more_rows_of_one_expert_than_a_token_list(T, E, D, F):
    """The weight gradients list 4096 tokens at a time: an expert with more of them."""
    col, val = routing(T, E, 1, 13, hot=0.97)
    assert int((col == 0).sum()) > 4096
    x, w_in, w_out, dy = tensors(T, E, D, F, BF, 14)
    print(f"T={T} E={E} D={D} F={F}", flush=True)
    want = ref.experts(x, w_in, w_out, col, val, dy)
    _, kept = sg.experts(*(t.cuda() for t in (x, w_in, w_out, col, val)), keep=True)
    got = sg.experts_backward(dy.cuda(), kept)
    torch.cuda.synchronize()
    for name, g in zip(("grad_x", "grad_w_in", "grad_w_out", "grad_val"), got):
        ref.assert_within(g, *want[name], name)


def test_strided_and_unaligned_operands():
    T, E, k, D, F = 37, 5, 2, 64, 48
    col, val = routing(T, E, k, 1)
    x, w_in, w_out, dy = tensors(T, E, D, F, BF, 2)
    want = ref.experts(x, w_in, w_out, col, val, dy)
    for ld, off in ((D + 8, 0), (D + 3, 0), (D, 1), (D + 8, 5)):
        def strided(t):
            buf = torch.full((T * ld + off + 8,), float("nan"), dtype=BF, device="cuda")
            v = buf[off:off + T * ld].view(T, ld)[:, :D]
            v.copy_(t.cuda())
            return v
        def shifted(t):
            buf = torch.empty(t.numel() + off, dtype=BF, device="cuda")
            v = buf[off:].view(t.shape)
            v.copy_(t.cuda())
            return v
        print(f"stride {ld}, offset {off}", flush=True)
        y, kept = sg.experts(strided(x), shifted(w_in), shifted(w_out), col.cuda(), val.cuda(),
                             keep=True)
        got = sg.experts_backward(strided(dy), kept)
        torch.cuda.synchronize()
        ref.assert_within(y, *want["y"], "y")
        for name, g in zip(("grad_x", "grad_w_in", "grad_w_out", "grad_val"), got):
            ref.assert_within(g, *want[name], name)


@pytest.mark.parametrize("T,E,k", [(600, 2, 2), (560, 8, 1)])
def test_rows_spread_over_more_than_4_gb(T, E, k):
    """Row strides whose byte offsets pass 32 bits, for x and for the gradient of y."""
    D, F, ld = 40, 24, 1 << 22
    print(f"far rows T={T} E={E}: {T * ld * 2 / 2 ** 30:.1f} GiB between the first and the last", flush=True)
    col, val = routing(T, E, k, 11)
    x, w_in, w_out, dy = tensors(T, E, D, F, BF, 12)
    want = ref.experts(x, w_in, w_out, col, val, dy)
    buf = torch.empty(T * ld, dtype=BF, device="cuda").view(T, ld)
    x_far, dy_far = buf[:, :D], buf[:, 64:64 + D]
    x_far.copy_(x.cuda())
    dy_far.copy_(dy.cuda())
    args = w_in.cuda(), w_out.cuda(), col.cuda(), val.cuda()
    y, kept = sg.experts(x_far, *args, keep=True)
    got = sg.experts_backward(dy_far, kept)
    few = sg.experts(x_far[-2:], *args[:2], args[2][-2:].contiguous(), args[3][-2:].contiguous())
    torch.cuda.synchronize()
    ref.assert_within(y, *want["y"], "y")
    ref.assert_within(few, want["y"][0][-2:], want["y"][1][-2:], "y of the last two")
    for name, g in zip(("grad_x", "grad_w_in", "grad_w_out", "grad_val"), got):
        ref.assert_within(g, *want[name], name)


def test_gradients_against_differences():
    """The gradients' definition (the oracle's) against central differences of the layer in fp64."""
    T, E, k, D, F = 6, 3, 2, 10, 6
    col, val = routing(T, E, k, 3)
    x, w_in, w_out, dy = (t.double() for t in tensors(T, E, D, F, HF, 4))
    def layer(x, w_in, w_out, val):
        y = torch.zeros_like(x)
        for t in range(T):
            for i in range(k):
                e = int(col[t, i])
                p = w_in[e] @ x[t]
                y[t] += val[t, i] * (w_out[e] @ (torch.nn.functional.silu(p[:F]) * p[F:]))
        return (y * dy).sum()
    half = [t.to(HF) for t in (x, w_in, w_out)]
    want = ref.experts(*half, col, val, dy.to(HF))
    got = sg.experts(*(t.cuda() for t in half), col.cuda(), val.cuda(), keep=True)[1]
    got = sg.experts_backward(dy.to(HF).cuda(), got)
    torch.cuda.synchronize()
    args = [x, w_in, w_out, val.double()]
    for n, (at, name) in enumerate(zip(args, ("grad_x", "grad_w_in", "grad_w_out", "grad_val"))):
        value, bound = want[name]
        rng = np.random.default_rng(n)
        for _ in range(8):
            j = tuple(int(rng.integers(s)) for s in at.shape)
            step = 1e-5
            up, down = [a.clone() for a in args], [a.clone() for a in args]
            up[n][j] += step
            down[n][j] -= step
            num = float(layer(*up) - layer(*down)) / (2 * step)
            assert abs(num - float(value[j])) <= 1e-6 * (1 + abs(num)), (name, j)
            assert abs(float(got[n][j]) - num) <= float(bound[j]) + 1e-6 * (1 + abs(num)), (name, j)


def test_no_tokens():
    E, D, F = 3, 16, 8
    _, w_in, w_out, _ = tensors(1, E, D, F, BF, 0)
    x = torch.empty(0, D, dtype=BF, device="cuda")
    col = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    val = torch.empty(0, 2, dtype=torch.float32, device="cuda")
    y, kept = sg.experts(x, w_in.cuda(), w_out.cuda(), col, val, keep=True)
    gx, gi, go, gv = sg.experts_backward(x, kept)
    torch.cuda.synchronize()
    assert y.shape == (0, D) and gx.shape == (0, D) and gv.shape == (0, 2)
    assert not bool(gi.any()) and not bool(go.any())
    row_ptr, entry = sg.dispatch(col, E)
    assert row_ptr.tolist() == [0] * (E + 1) and entry.numel() == 0


def test_columns_outside_are_no_entries():
    T, E, k, D, F = 9, 3, 2, 16, 8
    col, val = routing(T, E, k, 5)
    x, w_in, w_out, dy = tensors(T, E, D, F, BF, 6)
    bad = col.clone()
    bad[2, 1], bad[4, 0], bad[5, 1] = E, 2 ** 31 - 1, -7
    mask = (bad >= 0) & (bad < E)
    want = ref.experts(x, w_in, w_out, torch.where(mask, bad, -1), torch.where(mask, val, 0.0), dy)
    y, kept = sg.experts(x.cuda(), w_in.cuda(), w_out.cuda(), bad.cuda(), val.cuda(), keep=True)
    got = sg.experts_backward(dy.cuda(), kept)
    torch.cuda.synchronize()
    ref.assert_within(y, *want["y"], "y")
    for name, g in zip(("grad_x", "grad_w_in", "grad_w_out", "grad_val"), got):
        ref.assert_within(g, *want[name], name)


def test_rows_do_not_leak():
    """Infinities of one token stay in its own row, and those of rows without entries nowhere."""
    T, E, k, D, F = 70, 3, 1, 64, 32
    col, val = routing(T, E, k, 7)
    col[11, 0] = -1
    x, w_in, w_out, _ = tensors(T, E, D, F, BF, 8)
    clean = sg.experts(x.cuda(), w_in.cuda(), w_out.cuda(), col.cuda(), val.cuda()).cpu()
    x[11], x[30] = float("nan"), float("inf")
    y = sg.experts(x.cuda(), w_in.cuda(), w_out.cuda(), col.cuda(), val.cuda()).cpu()
    same = torch.ones(T, dtype=torch.bool)
    same[30] = False
    assert torch.equal(y[same], clean[same]) and bool((y[11] == 0).all())
    assert not bool(torch.isfinite(y[30]).all())


@pytest.mark.parametrize("T,E,k,idle", [(1, 1, 1, 0), (5, 3, 3, 0), (100, 17, 4, 0.2),
                                        (4095, 64, 1, 0), (4097, 60, 1, 0.1), (3000, 256, 8, 0.05),
                                        (700, 1024, 64, 0), (20000, 5, 2, 0)])
def test_dispatch_is_the_transpose(T, E, k, idle):
    print(f"dispatch T={T} E={E} k={k}", flush=True)
    rng = np.random.default_rng(T)
    col = rng.random((T, E)).argsort(1)[:, :k].astype(np.int32) if E * T < 3e6 else \
        rng.integers(0, E, (T, k)).astype(np.int32)
    col.sort(axis=1)
    col[rng.random(T) < idle] = -1
    row_ptr, entry = sg.dispatch(torch.from_numpy(col).cuda(), E)
    torch.cuda.synchronize()
    flat = col.reshape(-1)
    want = [np.flatnonzero(flat == e) for e in range(E)]
    assert row_ptr.cpu().tolist() == [0] + np.cumsum([len(w) for w in want]).tolist()
    n = int(row_ptr[-1])
    assert np.array_equal(entry.cpu().numpy()[:n], np.concatenate(want))


def test_another_stream_and_a_graph():
    T, E, k, D, F = 24, 4, 2, 64, 32
    col, val = routing(T, E, k, 9)
    x, w_in, w_out, dy = tensors(T, E, D, F, BF, 10)
    dev = [t.cuda() for t in (x, w_in, w_out, col, val)]
    dyc = dy.cuda()
    def step():
        y, kept = sg.experts(*dev, keep=True)
        return (y, *sg.experts_backward(dyc, kept), sg.clip_grad_norm([y], 1.0, out=[torch.empty_like(y)]))
    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        dev[0].mul_(-1.0)
        eager = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, eager):
            assert torch.equal(a, b), f"replay {i}"


def test_refusals():
    T, E, k, D, F = 4, 3, 2, 16, 8
    col, val = (t.cuda() for t in routing(T, E, k, 0))
    x, w_in, w_out, dy = (t.cuda() for t in tensors(T, E, D, F, BF, 0))
    for bad in (dict(x=x.float()), dict(x=x.cpu()), dict(x=x.t()), dict(w_in=w_in.to(HF)),
                dict(w_out=w_out.transpose(1, 2)), dict(col=col.long()), dict(val=val.to(BF)),
                dict(w_in=w_in[:, :-1].contiguous()), dict(val=val[:, :1].contiguous()),
                dict(x=x[:, :8])):
        args = dict(x=x, w_in=w_in, w_out=w_out, col=col, val=val) | bad
        with pytest.raises((TypeError, ValueError)):
            sg.experts(**args)
    _, kept = sg.experts(x, w_in, w_out, col, val, keep=True)
    for g in (dy[:-1], dy.float(), dy.cpu()):
        with pytest.raises((TypeError, ValueError)):
            sg.experts_backward(g, kept)
    wide = torch.zeros(1, 65, dtype=torch.int32, device="cuda")
    with pytest.raises(sg.SpgemmError) as e:
        sg.experts(x[:1], w_in, w_out, wide, wide.float())
    assert e.value.status == -1
    torch.cuda.synchronize()
