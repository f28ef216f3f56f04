"""Tensors that carry a tangent of torch's forward mode: the calls make no tangents, so they
refuse them, before anything that needs a GPU."""
import pytest

torch = pytest.importorskip("torch")
import torch.autograd.forward_ad as fwd

import spgemm_symbolic_row_amd as sg
from spgemm_symbolic_row_amd import expert_layer, norm

BF, E4 = torch.bfloat16, torch.float8_e4m3fn
T, E, D, F, k = 4, 8, 32, 16, 2


def r(*s, dtype=BF):
    return torch.ones(*s).to(dtype)


def calls():
    """(name, function of its tensors, the tensors)"""
    col, val = torch.zeros(T, k, dtype=torch.int32), r(T, k, dtype=torch.float32)
    routing = sg.Routing(col, val, E, None)
    x, w_in, w_out = r(T, D), r(E, 2 * F, D), r(E, D, F)
    scales = r(E, 1, 1, dtype=torch.float32)
    yield "layer_norm", sg.layer_norm, (x, r(D), r(D))
    yield "layer_norm_backward", lambda g: sg.layer_norm_backward(
        g, norm._KeptRows(x, r(D), False, (T, D), BF, 1e-5, 1, None, 0)), (x,)
    yield "experts", lambda x, a, b, v: sg.experts(x, a, b, col, v), (x, w_in, w_out, val)
    yield "experts, kept in 8 bits", lambda x, a, b, v: sg.experts(x, a, b, col, v, keep="e4m3"), (x, w_in, w_out, val)
    yield "experts_backward", lambda g: sg.experts_backward(
        g, expert_layer._Kept(x, w_in, w_out, val, None, 0)), (x,)
    yield "route", lambda z: sg.route(z, k), (r(T, E),)
    yield "route_backward", lambda z, g: sg.route_backward(z, routing, g), (r(T, E), val)
    yield "expert_step", lambda *t: sg.expert_step(*t, k), (x, r(E, D), w_in, w_out)
    yield "expert_step, 8 bits", lambda x, p, s, t: sg.expert_step(
        x, p, w_in.to(E4), w_out.to(E4), k, in_scale=s, out_scale=t), (x, r(E, D), scales, scales.clone())
    yield "clip_grad_norm", lambda *g: sg.clip_grad_norm(g, 1.0), (x, val)


@pytest.mark.parametrize("name,f,tensors", [pytest.param(*c, id=c[0]) for c in calls()])
def test_tangents_are_refused(name, f, tensors):
    for i in range(len(tensors)):
        with fwd.dual_level():
            given = [fwd.make_dual(t, torch.ones_like(t)) if j == i else t for j, t in enumerate(tensors)]
            for mode in (torch.enable_grad, torch.no_grad):
                with mode(), pytest.raises(TypeError, match="tangent"):
                    f(*given)
            # Beside other work in forward mode, tensors without a tangent get as far as the device.
            with pytest.raises(TypeError, match="device"):
                f(*(fwd.unpack_dual(t).primal for t in given))
    with pytest.raises(TypeError, match="device"):
        f(*tensors)
