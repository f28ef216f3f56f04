"""A block as a model has it, x + experts(layer_norm(x)): its forward and backward pass in
training, with everything kept in 8 bits, and the same weights served for a few
tokens.  Each step is held to its own 64-bit form, from what the step before gave."""
import pytest

torch = pytest.importorskip("torch")
sg = pytest.importorskip("spgemm_symbolic_row_amd")
import expert_reference as ref
import norm_reference as norm_ref
import rows8_reference as rows8
from expert_reference import assert_within

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def block(T, E, k, D, F, dtype, keep):
    gen = torch.Generator().manual_seed(T + D)
    def r(*s, scale=1.0):
        return (torch.randn(*s, generator=gen) * scale)
    host = dict(x=r(T, D, scale=2.0).to(dtype), g=(1 + 0.2 * r(D)), b=0.1 * r(D), router=r(E, D, scale=D ** -0.5),
                w_in=r(E, 2 * F, D, scale=D ** -0.5).to(dtype), w_out=r(E, D, F, scale=F ** -0.5).to(dtype),
                dy=r(T, D).to(dtype))
    d = {n: v.cuda() for n, v in host.items()}
    h, kept_norm = sg.layer_norm(d["x"], d["g"], d["b"], keep=keep)
    logits = (h.double() @ d["router"].double().t()).float()
    routing = sg.route(logits, k)
    y, kept = sg.experts(h, d["w_in"], d["w_out"], routing.col, routing.val, keep=keep)
    dh, dw_in, dw_out, dval = sg.experts_backward(d["dy"], kept)
    dlogits = sg.route_backward(logits, routing, dval)
    dh = (dh.float() + dlogits @ d["router"]).to(dtype)
    dx, dg, db = sg.layer_norm_backward(dh, kept_norm)
    out = dict(h=h, col=routing.col, val=routing.val, y=y, dw_in=dw_in, dw_out=dw_out, dval=dval, dh=dh, dx=dx, dg=dg, db=db)
    torch.cuda.synchronize()
    return host, d, {n: v.cpu() for n, v in out.items()}


@pytest.mark.parametrize("T,E,k,D,F,dtype", [(16, 8, 2, 256, 72, BF), (200, 5, 2, 136, 64, HF), (33, 16, 3, 101, 40, BF)])
@pytest.mark.parametrize("keep", [True, "e4m3"])
def test_training_step(T, E, k, D, F, dtype, keep):
    host, _, got = block(T, E, k, D, F, dtype, keep)
    at = rows8.kept(host["x"]) if keep == "e4m3" else None
    want = norm_ref.layer_norm(host["x"], host["g"], host["b"], 1e-5, got["dh"], at)
    assert_within(got["h"], *want["y"], "h")
    for name, mine in (("grad_x", "dx"), ("grad_weight", "dg"), ("grad_bias", "db")):
        assert_within(got[mine], *want[name], mine)
    h = got["h"]
    assert_within(got["y"], *ref.experts(h, host["w_in"], host["w_out"], got["col"], got["val"])["y"], "y")
    if keep == "e4m3":
        h = rows8.kept(h).to(dtype)
    want = ref.experts(h, host["w_in"], host["w_out"], got["col"], got["val"], host["dy"])
    for name, mine in (("grad_w_in", "dw_in"), ("grad_w_out", "dw_out"), ("grad_val", "dval")):
        assert_within(got[mine], *want[name], mine)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_serving_gives_what_training_gave(dtype):
    """The same rows through the layer for a few tokens: the same picks, and y within both bounds."""
    T, E, k, D, F = 16, 8, 2, 256, 72
    host, d, got = block(T, E, k, D, F, dtype, True)
    bound = ref.experts(got["h"], host["w_in"], host["w_out"], got["col"], got["val"])["y"][1]
    for rows in (slice(0, 1), slice(3, 8), slice(0, 16)):
        h = sg.layer_norm(d["x"][rows], d["g"], d["b"])
        assert torch.equal(h.cpu(), got["h"][rows])
        y, r = sg.expert_step(h, d["router"], d["w_in"], d["w_out"], k)
        torch.cuda.synchronize()
        assert torch.equal(r.col.cpu(), got["col"][rows])
        # The values differ by the order of their sums, 2^-18 of them at most, and so does y on top of both bounds.
        assert bool(((r.val.cpu() - got["val"][rows]).abs() <= 2.0 ** -18 * got["val"][rows]).all())
        size = ref.experts(got["h"].abs(), host["w_in"].abs(), host["w_out"].abs(), got["col"], got["val"])["y"][0]
        slack = 2 * bound + 2.0 ** -18 * size
        assert bool(((y.cpu().double() - got["y"][rows].double()).abs() <= slack[rows]).all())
