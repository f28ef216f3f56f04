"""Routing and its gradient against a plain form row by row in 64 bits.

Keys are fp32 by definition, so the columns have to be equal.  Bounds of the
values: exp and division within 2^-20 relative, sums of at most E fp32 terms
within E 2^-23; the gradients add differences of such terms, so theirs are
relative to the largest product in the row; 16-bit gradients add a rounding."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
sg = pytest.importorskip("spgemm_symbolic_row_amd")
import expert_reference as ref

pytestmark = pytest.mark.gpu

F32, BF, HF = torch.float32, torch.bfloat16, torch.float16
HALF_ULP = {F32: 2.0 ** -24, BF: 2.0 ** -8, HF: 2.0 ** -11}
INF = float("inf")


def check(logits, k, grad=True, strided=None, **how):
    T, E = logits.shape
    gen = torch.Generator().manual_seed(T * 31 + E)
    dv = torch.randn(T, k, generator=gen) if grad else None
    col, val, dz = ref.route(logits, k, grad=dv, **how)
    dev = {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in how.items()}
    z = logits.cuda() if strided is None else strided(logits)
    r = sg.route(z, k, **dev)
    got = sg.route_backward(z, r, dv.cuda()) if grad else None
    torch.cuda.synchronize()
    assert torch.equal(r.col.cpu(), col), torch.nonzero(r.col.cpu() != col)[:3]
    tol = 4 * 2.0 ** -20 + E * 2.0 ** -22
    ref.assert_within(r.val, val, tol * val.abs() + 1e-37, "val")
    if grad:
        assert got.dtype == logits.dtype
        scale = how.get("scale", 1.0) * dv.abs().amax(1, keepdim=True).double()
        bound = 8 * tol * scale.expand_as(dz) + HALF_ULP[logits.dtype] * dz.abs() + 2.0 ** -25
        ref.assert_within(got, dz, bound, "grad_logits")
    return r


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,dtype,how", [
    (1, 1, 1, F32, {}),
    (1, 64, 6, BF, {}),
    (7, 8, 8, HF, dict(renormalise=False)),
    (37, 60, 4, BF, dict(renormalise=False, bias=True)),
    (50, 65, 9, F32, dict(bias=True, scale=2.5)),
    (33, 128, 64, HF, {}),
    (21, 256, 8, F32, dict(groups=8, top_groups=4, bias=True, scale=2.5)),
    (21, 254, 5, BF, dict(groups=2, top_groups=1)),
    (19, 63, 3, F32, dict(groups=21, top_groups=2, bias=True)),
    (19, 64, 2, BF, dict(groups=64, top_groups=7)),
    (11, 300, 10, F32, dict(groups=3, top_groups=2, renormalise=False)),
    (9, 512, 20, BF, dict(groups=4, top_groups=4)),
    (5, 1024, 32, F32, dict(bias=True)),
    (5, 1021, 3, HF, {}),
])
def test_route(T, E, k, dtype, how, scores):
    print(f"route T={T} E={E} k={k} {dtype} {scores} {how}", flush=True)
    gen = torch.Generator().manual_seed(E + T)
    logits = torch.randn(T, E, generator=gen).mul_(1.5).to(dtype)
    how = dict(how)
    if how.get("bias"):
        how["bias"] = torch.randn(E, generator=gen) * 0.1
    if T > 5:
        how["active"] = torch.rand(T, generator=gen) > 0.2
    check(logits, k, scores=scores, **how)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_masked_rows_ties_and_extremes(scores, groups):
    E, k = 16, 4
    rows = [torch.zeros(E), torch.full((E,), -INF), torch.full((E,), -3.4e38),
            torch.linspace(-100, 100, E), torch.linspace(100, -100, E),
            torch.full((E,), -90.0), torch.tensor([0.0, -0.0] * 8)]
    one = torch.full((E,), -INF)
    one[9] = 1.0
    two = one.clone()
    two[3] = 1.0
    ties = torch.tensor([1.0, 2.0, 2.0, 1.0] * 4)
    low = torch.full((E,), -3.4e38)
    low[5] = 3.0
    z = torch.stack(rows + [one, two, ties, low])
    check(z, k, scores=scores, groups=groups, top_groups=2 if groups > 1 else 0)
    check(z, k, scores=scores, renormalise=False)


def test_masked_places_may_hold_anything():
    """NaN logits are out; rows that are not active are not looked at; a bias of -inf takes an expert out."""
    E, k, T = 24, 3, 6
    gen = torch.Generator().manual_seed(0)
    z = torch.randn(T, E, generator=gen)
    z[1, 4:9] = float("nan")
    z[2] = float("nan")
    active = torch.ones(T, dtype=torch.bool)
    active[2] = active[3] = False
    z[3, ::2] = INF
    bias = torch.zeros(E)
    bias[[0, 7]] = -INF
    for how in (dict(), dict(renormalise=False), dict(scores="sigmoid")):
        r = check(z, k, bias=bias, active=active, **how)
        assert bool((r.col.cpu()[2:4] == -1).all()) and bool((r.val.cpu()[2:4] == 0).all())
        assert not bool(torch.isnan(r.val).any())


def test_strides_and_offsets():
    T, E, k = 13, 40, 4
    z = torch.randn(T, E, generator=torch.Generator().manual_seed(3))
    for dtype in (F32, BF):
        for ld, off in ((E + 4, 0), (E + 1, 0), (E, 1), (E + 24, 3)):
            def strided(t):
                buf = torch.full((T * ld + off + 8,), float("nan"), dtype=dtype, device="cuda")
                v = buf[off:off + T * ld].view(T, ld)[:, :E]
                v.copy_(t.cuda())
                return v
            check(z.to(dtype), k, strided=strided)
            check(z.to(dtype)[:, :E], k, strided=strided, renormalise=False)


@pytest.mark.parametrize("how", [dict(), dict(renormalise=False), dict(scores="sigmoid"),
                                 dict(scores="sigmoid", renormalise=False, scale=1.7)])
def test_gradient_against_differences(how):
    """The oracle's gradient against central differences of its values, in 64 bits."""
    T, E, k = 4, 12, 3
    gen = torch.Generator().manual_seed(5)
    z = torch.randn(T, E, generator=gen).double()
    dv = torch.randn(T, k, generator=gen)
    r = sg.route(z.float().cuda(), k, **how)
    got = sg.route_backward(z.float().cuda(), r, dv.cuda()).cpu().double()
    z = z.float().double()
    col = r.col.cpu().long()
    def value(z):
        if how.get("scores") == "sigmoid":
            p = torch.sigmoid(z).gather(1, col)
            w = p if not how.get("renormalise", True) else p / (p.sum(1, keepdim=True) + 1e-20)
        elif how.get("renormalise", True):
            w = torch.softmax(z.gather(1, col), 1)
        else:
            w = torch.softmax(z, 1).gather(1, col)
        return float((w * how.get("scale", 1.0) * dv.double()).sum())
    for t in range(T):
        for e in range(E):
            up, down = z.clone(), z.clone()
            up[t, e] += 1e-5
            down[t, e] -= 1e-5
            assert abs((value(up) - value(down)) / 2e-5 - float(got[t, e])) < 2e-5


def test_no_tokens_and_csr():
    r = sg.route(torch.empty(0, 8, device="cuda"), 2)
    assert r.col.shape == (0, 2) and r.val.shape == (0, 2)
    # R^T R counts the tokens that two experts share.
    T, E, k = 200, 12, 3
    z = torch.randn(T, E, generator=torch.Generator().manual_seed(1))
    z[5] = -INF
    r = sg.route(z.cuda(), k)
    R = r.csr()
    row_ptr, entry = sg.dispatch(r.col, E)
    Rt = sg.transpose(R)
    assert torch.equal(Rt.row_ptr, row_ptr)
    n = int(row_ptr[-1])
    assert torch.equal(Rt.col, torch.div(entry[:n], k, rounding_mode="floor").int())
    R.val = torch.ones_like(R.val)
    Rt.val = torch.ones_like(R.val)
    rp, c, v = sg.matmul(Rt, R)
    torch.cuda.synchronize()
    full = torch.zeros(T, E)
    for t in range(T):
        for e in r.col[t].cpu():
            if e >= 0:
                full[t, e] = 1
    want = full.T @ full
    rows = torch.repeat_interleave(torch.arange(E), rp.cpu().diff())
    got = torch.zeros(E, E)
    got[rows, c.cpu().long()] = v.cpu()
    assert torch.equal(got, want)


def test_refusals():
    z = torch.zeros(4, 16, device="cuda")
    ok = torch.zeros(16, device="cuda")
    for args, how in (((z.cpu(), 2), {}), ((z.double(), 2), {}), ((z.t(), 2), {}), ((z[0], 2), {}),
                      ((z, 2), dict(scores="max")), ((z, 2), dict(scale=0.0)),
                      ((z, 2), dict(bias=ok[:-1])), ((z, 2), dict(bias=ok.half())),
                      ((z, 2), dict(active=ok[:4])), ((z, 2), dict(groups=0))):
        with pytest.raises((TypeError, ValueError)):
            sg.route(*args, **how)
    for k, how in ((0, {}), (17, {}), (-1, {}), (2, dict(groups=3)), (2, dict(groups=4, top_groups=5)),
                   (5, dict(groups=4, top_groups=1))):
        with pytest.raises(sg.SpgemmError) as e:
            sg.route(z, k, **how)
        assert e.value.status == -1
    with pytest.raises(sg.SpgemmError):
        sg.route(torch.zeros(1, 1025, device="cuda"), 2)
    r = sg.route(z, 2)
    with pytest.raises(ValueError):
        sg.route_backward(z[:3], r, torch.zeros(3, 2, device="cuda"))
    with pytest.raises(ValueError):
        sg.route_backward(z, r, torch.zeros(4, 3, device="cuda"))
    with pytest.raises(TypeError):
        sg.route_backward(z, r, torch.zeros(4, 2, dtype=BF, device="cuda"))
    torch.cuda.synchronize()


@pytest.mark.parametrize("k,renormalise", [(1, False), (3, False), (3, True)])
def test_slope_of_a_saturated_sigmoid(k, renormalise):
    """The slope s (1 - s) at large logits, where 1 - s has few bits left: every gradient to a
    relative bound.  With z at +-12 .. +-80, exp and its argument are off by 2^-22 + |z| 2^-24 <=
    2^-17, the rest by 2^-20; renormalised, a difference of two terms is held to their size."""
    z = torch.tensor([[12.0, -12.0, 20.0], [-20.0, 17.0, 30.0], [-80.0, 80.0, 40.0],
                      [0.5, -40.0, 16.6]])[:, :k].contiguous()
    dv = torch.tensor([[1.0, -2.0, 0.5]])[:, :k].repeat(4, 1).contiguous()
    r = sg.route(z.cuda(), k, scores="sigmoid", renormalise=renormalise)
    got = sg.route_backward(z.cuda(), r, dv.cuda())
    torch.cuda.synchronize()
    s, e = torch.sigmoid(z.double()), torch.exp(-z.double().abs())
    d, size = dv.double(), dv.double().abs()
    if renormalise:
        total = s.sum(1, keepdim=True) + 1e-20
        mean = (s * d).sum(1, keepdim=True) / total
        size = (size + (s * size).sum(1, keepdim=True) / total) / total
        d = (d - mean) / total
    slope = e / (1 + e) ** 2
    ref.assert_within(got, d * slope, 2.0 ** -16 * size * slope + 1e-37, "grad_logits")


def test_more_rows_than_one_launch_takes():
    """A launch has fewer than 2^32 work items: 16 or 64 to a row of logits."""
    T = (1 << 28) + 1003
    z = torch.zeros(T, 1, dtype=BF, device="cuda")
    r = sg.route(z, 1)
    assert int(torch.count_nonzero(r.col)) == 0 and float(r.val.min()) == 1.0 == float(r.val.max())
    del z, r
    T, E, k = (1 << 26) + 77, 3, 2
    z = torch.randn(T, E, dtype=BF, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    active = torch.rand(T, device="cuda") > 0.1
    r = sg.route(z, k, active=active)
    g = torch.randn(T, k, device="cuda")
    dz = sg.route_backward(z, r, g)
    for part in (slice(0, 999), slice((1 << 25) - 50, (1 << 25) + 50), slice(T - 999, T)):
        q = sg.route(z[part], k, active=active[part])
        assert torch.equal(q.col, r.col[part]) and torch.equal(q.val, r.val[part])
        assert torch.equal(sg.route_backward(z[part], q, g[part]), dz[part])
    torch.cuda.synchronize()
