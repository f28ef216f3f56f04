"""expert_step and layer norm in captured graphs that run two calls at once, or share their
memory with another graph."""
import pytest

torch = pytest.importorskip("torch")
sg = pytest.importorskip("spgemm_symbolic_row_amd")
from test_gpu_step import BF, E4, tensors

pytestmark = pytest.mark.gpu

T, E, k, D, F = 16, 32, 4, 520, 264


def state(i, wdtype):
    g = [None if v is None else v.cuda() for v in tensors(T, E, D, F, BF, wdtype, BF, 40 + i)]
    w = torch.randn(D, device="cuda")

    def block():
        h, kept = sg.layer_norm(g[0], w, w, keep="e4m3")
        y, r = sg.expert_step(h, *g[1:4], k, in_scale=g[4], out_scale=g[5])
        return (y, r.col, r.val, *sg.layer_norm_backward(y, kept))
    return g[0], block


def replays(graphs, states, outs):
    for i in range(4):
        for x, _ in states:
            x.copy_(torch.randn(T, D, device="cuda"))
        for graph, which in graphs:
            graph.replay()
            got = [[t.clone() for t in outs[j]] for j in which]
            torch.cuda.synchronize()
            for j, a in zip(which, got):
                assert all(torch.equal(p, q) for p, q in zip(a, states[j][1]())), (i, j)


def captured(work, pool=None):
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, pool=pool):
        outs = work()
    return graph, outs


def test_two_calls_at_once_in_a_graph():
    states = [state(0, BF), state(1, E4)]
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        for _, block in states:
            block()

    def both():
        main = torch.cuda.current_stream()
        other.wait_stream(main)
        first = states[0][1]()
        with torch.cuda.stream(other):
            second = states[1][1]()
        main.wait_stream(other)
        return first, second
    graph, outs = captured(both)
    replays([(graph, (0, 1))], states, outs)


def test_two_graphs_that_share_memory():
    states = [state(2, E4), state(3, BF)]
    for _, block in states:
        block()
    one, a = captured(states[0][1])
    two, b = captured(states[1][1], one.pool())
    replays([(one, (0,)), (two, (1,))], states, [a, b])
