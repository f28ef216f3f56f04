"""expert_step and layer_norm where offsets pass 32 bits: an expert's weights, and rows of x."""
import pytest

torch = pytest.importorskip("torch")
sg = pytest.importorskip("spgemm_symbolic_row_amd")

pytestmark = pytest.mark.gpu

F32, BF, E4 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.mark.parametrize("wdtype", [BF, E4])
def test_weights_beyond_4_gb(wdtype):
    """Three of 1024 experts can be picked, the last among them; the same three as a layer of their own give the same
    bits, since sums go over the picked experts in their order."""
    T, E, k, D, F = 5, 1024, 2, 2048, 2100
    w_in = torch.empty(E, 2 * F, D, dtype=wdtype, device="cuda")
    w_out = torch.empty(E, D, F, dtype=wdtype, device="cuda")
    b = torch.empty(0, dtype=wdtype).element_size()
    at = [0, 700, 1023]
    assert at[1] * D * F * b > 2 ** 31 and at[2] * 2 * F * D * b > 2 ** 32 and at[2] * D * F * b > 2 ** 32
    gen = torch.Generator(device="cuda").manual_seed(1)
    def r(*s):
        return torch.randn(*s, generator=gen, device="cuda")
    for e in at:
        w_in[e] = (r(2 * F, D) * (D ** -0.5 if wdtype is BF else 50.0)).to(wdtype)
        w_out[e] = (r(D, F) * (F ** -0.5 if wdtype is BF else 50.0)).to(wdtype)
    up = lambda n: -(-n // 128)
    scales, some = {}, {}
    if wdtype is E4:
        s_in, s_out = r(E, up(2 * F), up(D)) * D ** -0.5 / 50, r(E, up(D), up(F)) * F ** -0.5 / 50
        scales = dict(in_scale=s_in, out_scale=s_out)
        some = dict(in_scale=s_in[at].contiguous(), out_scale=s_out[at].contiguous())
    x, router = r(T, D).to(BF), r(E, D) * D ** -0.5
    bias = torch.full((E,), float("-inf"), device="cuda")   # a key of minus infinity is out
    bias[at] = 0.0
    how = dict(scores="sigmoid", renormalise=False)          # a weight is its own expert's alone
    y, q = sg.expert_step(x, router, w_in, w_out, k, bias=bias, **scales, **how)
    part = lambda w: torch.stack([w[e].view(torch.uint8) for e in at]).view(wdtype)
    z, p = sg.expert_step(x, router[at].contiguous(), part(w_in), part(w_out), k, **some, **how)
    torch.cuda.synchronize()
    number = torch.tensor(at, device="cuda", dtype=torch.int32)
    assert torch.equal(q.col, number[p.col.long()]) and torch.equal(q.val, p.val)
    assert 1023 in q.col and bool(torch.isfinite(y).all()) and bool((y != 0).any())
    assert torch.equal(y, z)


def test_rows_beyond_4_gb():
    """The largest stride that is taken: the last rows begin beyond 2^32 bytes."""
    T, D, ld = 5, 136, 2 ** 30 - 1
    buf = torch.empty((T - 1) * ld + D, dtype=BF, device="cuda")
    far = buf.as_strided((T, D), (ld, 1))
    x = torch.randn(T, D, device="cuda").to(BF)
    far.copy_(x)
    w = torch.ones(D, device="cuda")
    for keep in (True, "e4m3"):
        y, kept = sg.layer_norm(x, w, w, keep=keep)
        z, kept_far = sg.layer_norm(far, w, w, keep=keep)
        assert torch.equal(y, z)
        for p, q in zip(sg.layer_norm_backward(x, kept), sg.layer_norm_backward(far, kept_far)):
            assert torch.equal(p, q)
    E, F = 4, 40
    router, w_in, w_out = (torch.randn(*s, device="cuda").to(BF) for s in ((E, D), (E, 2 * F, D), (E, D, F)))
    for t in (x, far):
        y, r = sg.expert_step(t, router, w_in, w_out, 2)
        if t is x:
            want, col = y, r.col
    assert torch.equal(y, want) and torch.equal(r.col, col)
    col, val = r.col, r.val
    a, b = (sg.experts(t, w_in, w_out, col, val, keep="e4m3") for t in (x, far))
    assert torch.equal(a[0], b[0])
    assert all(torch.equal(p, q) for p, q in zip(sg.experts_backward(x, a[1]), sg.experts_backward(far, b[1])))
    torch.cuda.synchronize()
