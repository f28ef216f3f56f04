"""The expert layer beside torch's own machinery: gradients that torch was to
make, streams, and counters of in-place changes."""
import pytest

torch = pytest.importorskip("torch")
sg = pytest.importorskip("spgemm_symbolic_row_amd")
from test_gpu_experts import routing, tensors

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def layer(T=4, E=3, k=2, D=16, F=8):
    col, val = routing(T, E, k, 0)
    x, w_in, w_out, dy = tensors(T, E, D, F, BF, 0)
    return [t.cuda() for t in (x, w_in, w_out, col, val)], dy.cuda()


def test_tensors_that_require_a_gradient_are_refused():
    """The calls record nothing for torch's backward pass, so a result without its graph would lose
    gradients silently."""
    args, dy = layer()
    plain = sg.experts(*args)
    for i in (0, 1, 2, 4):
        bad = list(args)
        bad[i] = args[i].clone().requires_grad_()
        with pytest.raises(TypeError, match="gradient"):
            sg.experts(*bad)
        with torch.no_grad():
            assert torch.equal(sg.experts(*bad), plain)
        assert torch.equal(sg.experts(*(t.detach() for t in bad)), plain)
    z = torch.randn(4, 8, device="cuda")
    bad = z.clone().requires_grad_()
    with pytest.raises(TypeError, match="gradient"):
        sg.route(bad, 2)
    with torch.no_grad():
        assert torch.equal(sg.route(bad, 2).col, sg.route(z, 2).col)
    # The bias enters the choice only: it has no gradient.
    assert torch.equal(sg.route(z, 2, bias=torch.zeros(8, device="cuda").requires_grad_()).col,
                       sg.route(z, 2).col)
    _, kept = sg.experts(*args, keep=True)
    with pytest.raises(TypeError, match="gradient"):
        sg.experts_backward(dy.clone().requires_grad_(), kept)
    r = sg.route(z, 2)
    with pytest.raises(TypeError, match="gradient"):
        sg.route_backward(z, r, torch.zeros(4, 2, device="cuda").requires_grad_())
    g = torch.ones(4, device="cuda")
    with pytest.raises(TypeError, match="gradient"):
        sg.clip_grad_norm([g], 1.0, out=[g.clone().requires_grad_()])
    torch.cuda.synchronize()


def test_clipping_counts_as_a_change():
    """Torch's check of tensors saved for a backward pass sees that they were clipped."""
    a, g = torch.ones(5, device="cuda", requires_grad=True), torch.full((5,), 3.0, device="cuda")
    y = (a * g).sum()   # saves g
    sg.clip_grad_norm([g], 1.0)
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward()
    g, o = torch.ones(5, device="cuda"), torch.ones(5, device="cuda")
    before = g._version, o._version
    sg.clip_grad_norm([g], 1.0, out=[o])
    assert g._version == before[0] and o._version > before[1]
    torch.cuda.synchronize()


def test_kept_block_outlives_a_backward_pass_on_another_stream():
    """What a forward pass kept is not given to its own stream again while a backward pass that
    another stream has yet to run reads it."""
    args, dy = layer(T=512, E=4, D=128, F=64)
    want = [t.clone() for t in sg.experts_backward(dy, sg.experts(*args, keep=True)[1])]
    torch.cuda.synchronize()
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    with torch.cuda.stream(side):
        _, kept = sg.experts(*args, keep=True)
    side.synchronize()
    at, size = kept.block.data_ptr(), kept.block.numel()
    torch.cuda._sleep(400_000_000)
    got = sg.experts_backward(dy, kept)
    del kept
    with torch.cuda.stream(side):
        new = torch.empty(size, dtype=torch.uint8, device="cuda")
    busy = not main.query()
    main.synchronize()
    assert busy and new.data_ptr() != at
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_an_error_that_another_call_left_is_not_reported():
    """The runtime keeps the last error of a thread until it is read."""
    args, dy = layer()
    z = torch.randn(4, 8, device="cuda")
    g = torch.ones(9, device="cuda")

    def every_call():
        left()
        r = sg.route(z, 2)
        left()
        d = sg.route_backward(z, r, r.val)
        left()
        p = sg.dispatch(r.col, 8)
        left()
        y, kept = sg.experts(*args, keep=True)
        left()
        b = sg.experts_backward(dy, kept)
        left()
        return (d, *p, y, *b, sg.clip_grad_norm([g], 1.0, out=[torch.empty_like(g)]))

    def left():
        pass

    want = every_call()
    torch.cuda.synchronize()
    hip = sg.lib()   # the runtime that the library is linked to

    def left():
        assert hip.hipSetDevice(1 << 20) != 0 and hip.hipPeekAtLastError() != 0

    got = every_call()
    hip.hipGetLastError()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("stride", [17, 1 << 30])
def test_stride_of_a_single_row(stride):
    """One token out of a larger tensor: whatever its row stride is, there is one row."""
    (x, w_in, w_out, col, val), dy = layer(T=1)
    def alone(t):
        v = torch.empty(stride + 64, dtype=t.dtype, device="cuda").as_strided(t.shape, (stride, 1))
        v.copy_(t)
        return v
    want, kept = sg.experts(x, w_in, w_out, col, val, keep=True)
    grads = sg.experts_backward(dy, kept)
    got, kept = sg.experts(alone(x), w_in, w_out, col, val, keep=True)
    assert torch.equal(got, want)
    assert all(torch.equal(a, b) for a, b in zip(sg.experts_backward(alone(dy), kept), grads))
    z = torch.randn(1, 8, device="cuda")
    assert torch.equal(sg.route(alone(z), 2).val, sg.route(z, 2).val)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,E", [(1, 3), (2, 16), (40, 16), (300, 3), (9000, 3)])
def test_no_row_has_an_entry(T, E, dtype):
    D, F, k = 72, 24, 2
    x, w_in, w_out, dy = (t.cuda() for t in tensors(T, E, D, F, dtype, 1))
    col = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    val = torch.full((T, k), float("nan"), device="cuda")
    y = sg.experts(x, w_in, w_out, col, val)
    z, kept = sg.experts(x, w_in, w_out, col, val, keep=True)
    for t in (y, z, *sg.experts_backward(dy, kept)):
        assert torch.count_nonzero(t) == 0
