"""A whole expert layer for a few tokens against a plain 64-bit form.

The logits' sums are made in 64 bits and rounded to fp32, so the columns have to be
equal; the values are held to the bounds of the routing's test, y to those of
expert_reference with the values that came out.  8-bit weights add one fp32
product and one addition for every 64 of a row's K products, which the reference's
2 K additions leave room for."""
import pytest

torch = pytest.importorskip("torch")
sg = pytest.importorskip("spgemm_symbolic_row_amd")
import expert_reference as ref

pytestmark = pytest.mark.gpu

F32, BF, HF, E4 = torch.float32, torch.bfloat16, torch.float16, torch.float8_e4m3fn


def spread(scale, rows, cols):
    return scale.double().repeat_interleave(128, 1)[:, :rows].repeat_interleave(128, 2)[:, :, :cols]


def tensors(T, E, D, F, dtype, wdtype, rdtype, seed):
    """x, router, w_in, w_out, in_scale, out_scale on the CPU."""
    gen = torch.Generator().manual_seed(seed)
    def r(*s, scale=1.0):
        return torch.randn(*s, generator=gen) * scale
    x, router = r(T, D).to(dtype), r(E, D, scale=1.5 * D ** -0.5).to(rdtype)
    if wdtype is not E4:
        return x, router, r(E, 2 * F, D, scale=D ** -0.5).to(dtype), r(E, D, F, scale=F ** -0.5).to(dtype), None, None
    up = lambda n: -(-n // 128)
    def weights(*s):
        return r(*s, scale=60.0).clamp(-448, 448).to(E4)
    return (x, router, weights(E, 2 * F, D), weights(E, D, F),
            r(E, up(2 * F), up(D)).abs().add(0.3) * (D ** -0.5 / 60), r(E, up(D), up(F)) * (F ** -0.5 / 60))


def reference(x, router, w_in, w_out, in_scale, out_scale, k, how):
    z = (x.double() @ router.double().t()).float()
    col, val, _ = ref.route(z, k, **how)
    if in_scale is not None:
        w_in = w_in.double() * spread(in_scale, *w_in.shape[1:])
        w_out = w_out.double() * spread(out_scale, *w_out.shape[1:])
    return col, val, w_in, w_out


def check(t, k, how=None, dev=None):
    how = how or {}
    x, router, w_in, w_out, in_scale, out_scale = t
    E = router.shape[0]
    col, val, wi, wo = reference(*t, k, how)
    g = [None if v is None else v.cuda() for v in t] if dev is None else dev
    opts = {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in how.items()}
    y, r = sg.expert_step(*g[:4], k, in_scale=g[4], out_scale=g[5], **opts)
    y2, _ = sg.expert_step(*g[:4], k, in_scale=g[4], out_scale=g[5], **opts)
    torch.cuda.synchronize()
    assert torch.equal(r.col.cpu(), col)
    ref.assert_within(r.val, val, (4 * 2.0 ** -20 + E * 2.0 ** -22) * val.abs() + 1e-37, "val")
    assert y.is_contiguous() and y.dtype == x.dtype and y.shape == x.shape
    ref.assert_within(y, *ref.experts(x, wi, wo, col, r.val.cpu())["y"], "y")
    assert torch.equal(y, y2)
    assert bool((y.cpu()[(col < 0).all(1)] == 0).all())
    return y, r


SIZES = [
    # T, E, k, D, F
    (1, 1, 1, 16, 16),
    (2, 3, 1, 17, 31),
    (3, 4, 2, 47, 79),
    (1, 4, 2, 64, 64),
    (1, 64, 6, 256, 128),
    (2, 8, 8, 63, 16),
    (3, 5, 2, 65, 17),
    (4, 24, 3, 100, 129),
    (5, 16, 2, 1001, 345),
    (7, 12, 4, 520, 63),
    (8, 3, 1, 130, 700),
    (9, 40, 5, 18, 16),
    (13, 60, 4, 264, 200),
    (16, 128, 8, 512, 96),
    (16, 2, 2, 2056, 72),
    (16, 300, 10, 72, 33),
    (6, 1024, 3, 40, 24),
    (16, 1024, 64, 16, 18),
    (1, 6, 2, 4104, 1032),
    (11, 16, 16, 128, 256),
    (10, 200, 6, 72, 40),
    (16, 4, 2, 4160, 48),    # rows of x that do not fit LDS
    (15, 3, 1, 4097, 40),
    (16, 5, 1, 8200, 33),
]


@pytest.mark.parametrize("wdtype", ["16-bit", "e4m3"])
@pytest.mark.parametrize("T,E,k,D,F", SIZES)
def test_layer(T, E, k, D, F, wdtype):
    dtype, rdtype = (BF, HF)[T % 2], F32 if E % 3 == 0 else (BF, HF)[T % 2]
    print(f"T={T} E={E} k={k} D={D} F={F} {dtype} {wdtype} router {rdtype}", flush=True)
    t = tensors(T, E, D, F, dtype, E4 if wdtype == "e4m3" else dtype, rdtype, T + E + D)
    check(t, k)


@pytest.mark.parametrize("wdtype", ["16-bit", "e4m3"])
def test_options_of_the_routing(wdtype):
    gen = torch.Generator().manual_seed(5)
    for T, E, k, how in ((16, 64, 4, dict(scores="sigmoid", groups=8, top_groups=3, scale=2.5, bias=True)),
                         (12, 60, 3, dict(renormalise=False, active=True)),
                         (9, 21, 2, dict(scores="sigmoid", renormalise=False, groups=7, top_groups=2)),
                         (16, 512, 20, dict(groups=4, top_groups=2, active=True, bias=True)),
                         (5, 8, 2, dict(active=True, scores="sigmoid"))):
        print(T, E, k, how, flush=True)
        if how.get("bias"):
            how["bias"] = torch.randn(E, generator=gen) * 0.1
        if how.get("active"):
            how["active"] = torch.rand(T, generator=gen) > 0.3
        for dtype in (BF, HF):
            check(tensors(T, E, 136, 72, dtype, E4 if wdtype == "e4m3" else dtype, F32, E), k, how)


def test_rows_that_are_not_routed_may_hold_anything():
    """And an expert that a token did not pick may hold anything, for that token."""
    T, E, k, D, F = 6, 8, 2, 200, 72
    for wdtype in (BF, E4):
        t = list(tensors(T, E, D, F, BF, wdtype, BF, 3))
        how = dict(active=torch.tensor([True, True, False, True, True, False]))
        want, r = check(t, k, how)
        bad = [None if v is None else v.clone() for v in t]
        bad[0][2], bad[0][5] = float("nan"), float("inf")
        g = [None if v is None else v.cuda() for v in bad]
        y, r2 = sg.expert_step(*g[:4], k, in_scale=g[4], out_scale=g[5], active=how["active"].cuda())
        assert torch.equal(y, want) and torch.equal(r.col, r2.col)
        lone = int(r.col[0, 0])
        for i in (2, 3):
            g[i][lone] = float("nan")
        y, _ = sg.expert_step(*g[:4], k, in_scale=g[4], out_scale=g[5], active=how["active"].cuda())
        hit = (r.col == lone).any(1)
        assert torch.equal(y[~hit], want[~hit]) and bool(torch.isnan(y[hit]).all()) and 0 < int(hit.sum()) < T
        # No row is routed; every logit is NaN.
        y, r2 = sg.expert_step(*g[:4], k, in_scale=g[4], out_scale=g[5],
                               active=torch.zeros(T, dtype=torch.bool, device="cuda"))
        assert torch.count_nonzero(y) == 0 and bool((r2.col == -1).all()) and torch.count_nonzero(r2.val) == 0
        g[0][:] = float("nan")
        y, r2 = sg.expert_step(*g[:4], k, in_scale=g[4], out_scale=g[5])
        assert torch.count_nonzero(y) == 0 and bool((r2.col == -1).all())


def test_close_experts_go_by_their_exact_logits():
    """Sums that cancel: 32 bits would lose what decides."""
    T, E, D, F = 3, 4, 2050, 16
    t = list(tensors(T, E, D, F, BF, BF, F32, 7))
    big = torch.randn(D // 2, generator=torch.Generator().manual_seed(1)) * 1e4
    for e in range(E):
        t[1][e, :D // 2], t[1][e, D // 2:] = big, -big
        t[1][e, 5] += 1e-3 * e
    t[0][:, D // 2:] = t[0][:, :D // 2]
    t[0][:, 5] = t[0][:, D // 2 + 5] = torch.tensor([1.0, -1.0, 2.0]).to(BF)
    _, r = check(t, 1)
    assert r.col[:, 0].tolist() == [3, 0, 3]


def test_ties_go_to_the_lowest_expert():
    t = list(tensors(5, 12, 64, 32, HF, HF, HF, 9))
    t[1][:] = t[1][0]
    _, r = check(t, 3)
    assert r.col.tolist() == [[0, 1, 2]] * 5


def test_strides_and_alignment():
    T, E, k, D, F = 5, 6, 2, 100, 40
    for wdtype in (HF, E4):
        t = tensors(T, E, D, F, HF, wdtype, HF, 11)
        for ld, off in ((D + 8, 0), (D + 3, 0), (D, 1), (D + 7, 5)):
            def shifted(v):
                buf = torch.zeros(v.numel() + off, dtype=v.dtype, device="cuda")
                buf[off:].copy_(v.reshape(-1))
                return buf[off:].view(v.shape)
            buf = torch.full((T * ld + off + 8,), float("nan"), dtype=HF, device="cuda")
            x = buf[off:off + T * ld].view(T, ld)[:, :D]
            x.copy_(t[0])
            check(t, k, dev=[x, *(None if v is None else shifted(v) for v in t[1:])])


@pytest.mark.parametrize("D", [4160, 4097])
def test_strides_of_rows_that_stay_in_memory(D):
    T, E, k, F = 16, 3, 2, 40
    for wdtype in (BF, E4):
        t = tensors(T, E, D, F, BF, wdtype, BF, 12)
        for ld, off in ((D + 8, 0), (D + 3, 1), (D, 1), (D + 2, 2)):
            buf = torch.full((T * ld + off + 8,), float("nan"), dtype=BF, device="cuda")
            x = buf[off:off + T * ld].view(T, ld)[:, :D]
            x.copy_(t[0])
            check(t, k, dev=[x, *(None if v is None else v.cuda() for v in t[1:])])


def test_an_error_that_another_call_left_is_not_reported():
    """The runtime keeps the last error of a thread until it is read."""
    t = [None if v is None else v.cuda() for v in tensors(4, 8, 64, 32, BF, BF, BF, 21)]
    w = torch.ones(64, device="cuda")
    hip = sg.lib()   # the runtime that the library is linked to

    def every_call(left):
        left()
        h, kept = sg.layer_norm(t[0], w, keep="e4m3")
        left()
        d = sg.layer_norm_backward(h, kept)[:2]
        left()
        return (h, *d, sg.expert_step(*t[:4], 2)[0])

    def left():
        assert hip.hipSetDevice(1 << 20) != 0 and hip.hipPeekAtLastError() != 0

    want = every_call(lambda: None)
    torch.cuda.synchronize()
    got = every_call(left)
    hip.hipGetLastError()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_stride_of_a_single_row():
    """One token out of a larger tensor: whatever its row stride is, there is one row."""
    t = [v.cuda() for v in tensors(1, 4, 64, 32, BF, BF, BF, 23)[:4]]
    w = torch.ones(64, device="cuda")
    want, norm = sg.expert_step(*t, 2)[0], sg.layer_norm(t[0], w)
    for stride in (17, 1 << 30):
        x = torch.empty(stride + 64, dtype=BF, device="cuda").as_strided((1, 64), (stride, 1))
        x.copy_(t[0])
        assert torch.equal(sg.expert_step(x, *t[1:], 2)[0], want)
        assert torch.equal(sg.layer_norm(x, w), norm)
    torch.cuda.synchronize()


def test_the_same_as_the_calls_that_it_joins():
    T, E, k, D, F = 16, 32, 4, 512, 256
    t = tensors(T, E, D, F, BF, BF, F32, 13)
    x, router, w_in, w_out = (v.cuda() for v in t[:4])
    y, r = check(t, k)
    q = sg.route((t[0].double() @ t[1].double().t()).float().cuda(), k)
    # Each value is within its bound; the sums of a row go over 16 lanes in one and 64 in the other.
    tol = 2 * (4 * 2.0 ** -20 + E * 2.0 ** -22)
    assert torch.equal(q.col, r.col) and bool(((q.val - r.val).abs() <= tol * q.val).all())
    z = sg.experts(x, w_in, w_out, r.col, r.val)
    bound = ref.experts(t[0], t[2], t[3], r.col.cpu(), r.val.cpu())["y"][1]
    assert bool(((y.double() - z.double()).abs().cpu() <= 2 * bound).all())


def test_graph_replays_and_streams():
    T, E, k, D, F = 8, 16, 3, 264, 136
    for wdtype in (BF, E4):
        g = [None if v is None else v.cuda() for v in tensors(T, E, D, F, BF, wdtype, BF, 15)]
        def step():
            y, r = sg.expert_step(*g[:4], k, in_scale=g[4], out_scale=g[5])
            return y, r.col, r.val
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        for i in range(5):
            g[0].copy_(torch.randn(T, D, device="cuda"))
            graph.replay()
            got = [v.clone() for v in out]
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, step())), i


def test_many_calls_at_once():
    """Calls on four streams, each with more work groups than the chip takes beside the others."""
    T, E, k, D, F = 16, 64, 8, 1024, 512
    calls = [[None if v is None else v.cuda() for v in tensors(T, E, D, F, BF, w, BF, 20 + i)]
             for i, w in enumerate((BF, E4, BF, E4))]
    def step(g):
        return sg.expert_step(*g[:4], k, in_scale=g[4], out_scale=g[5])[0]
    want = [step(g).clone() for g in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for _ in range(20):
        for i, (g, s) in enumerate(zip(calls, streams)):
            with torch.cuda.stream(s):
                got[i].append(step(g))
    torch.cuda.synchronize()
    for w, gs in zip(want, got):
        assert all(torch.equal(w, v) for v in gs)


def test_no_tokens_and_refusals():
    t = tensors(4, 8, 64, 32, BF, BF, BF, 17)
    x, router, w_in, w_out = (v.cuda() for v in t[:4])
    y, r = sg.expert_step(x[:0], router, w_in, w_out, 2)
    assert y.shape == (0, 64) and r.col.shape == (0, 2)
    q = tensors(4, 8, 64, 32, BF, E4, BF, 17)
    q_in, q_out, s_in, s_out = (v.cuda() for v in q[2:])
    def bad(error, *a, **k):
        with pytest.raises(error):
            sg.expert_step(*a, **k)
    bad(ValueError, x.repeat(5, 1)[:17], router, w_in, w_out, 2)
    bad(sg.SpgemmError, x, router, w_in, w_out, 0)
    bad(sg.SpgemmError, x, router, w_in, w_out, 9)
    bad(sg.SpgemmError, x, router, w_in, w_out, 2, groups=3)
    bad(ValueError, x, router, w_in, w_out, 2, scores="relu")
    bad(ValueError, x, router, w_in, w_out, 2, scale=0.0)
    bad(ValueError, x, router[:7], w_in, w_out, 2)
    bad(ValueError, x, router, w_in[:, :63], w_out, 2)
    bad(ValueError, x, router, w_in[0], w_out, 2)
    bad(TypeError, x, router.half(), w_in, w_out, 2)
    bad(TypeError, x, router, w_in.half(), w_out, 2)
    bad(TypeError, x, router, w_in.float(), w_out.float(), 2)
    bad(TypeError, x.float(), router, w_in, w_out, 2)
    bad(TypeError, x, router.cpu(), w_in, w_out, 2)
    bad(TypeError, x.cpu(), router, w_in, w_out, 2)
    bad(TypeError, x, router, w_in, q_out, 2, out_scale=s_out)
    bad(TypeError, x, router, q_in, w_out, 2, in_scale=s_in, out_scale=s_out)
    bad(ValueError, x, router, q_in, q_out, 2)
    bad(ValueError, x, router, q_in, q_out, 2, in_scale=s_in)
    bad(ValueError, x, router, w_in, w_out, 2, in_scale=s_in, out_scale=s_out)
    bad(ValueError, x, router, q_in, q_out, 2, in_scale=s_in[:, :, 1:], out_scale=s_out)
    bad(TypeError, x, router, q_in, q_out, 2, in_scale=s_in.half(), out_scale=s_out)
    bad(ValueError, x, router, w_in, w_out, 2, bias=torch.zeros(7, device="cuda"))
    bad(TypeError, x, router, w_in, w_out, 2, active=torch.ones(4, device="cuda"))
    for i in range(4):
        args = [x, router, w_in, w_out]
        args[i] = args[i].clone().requires_grad_()
        bad(TypeError, *args, 2)


def test_weights_in_8_bits_that_require_a_gradient():
    t = tensors(4, 8, 64, 32, BF, E4, BF, 17)
    given = [v.cuda() for v in t]
    for i in range(6):
        x, router, w_in, w_out, s_in, s_out = (v.clone().requires_grad_() if j == i else v
                                               for j, v in enumerate(given))
        with pytest.raises(TypeError, match="requires a gradient"):
            sg.expert_step(x, router, w_in, w_out, 2, s_in, s_out)
        with torch.no_grad():
            sg.expert_step(x, router, w_in, w_out, 2, s_in, s_out)
