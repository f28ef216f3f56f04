"""The expert-layer example runs its operators together: the loss falls, two runs
reach the same bits, and the routing matrix goes through the sparse product with
every token counted."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location(
        "expert_layer_example", os.path.join(ROOT, "examples", "expert_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_the_example_learns():
    m = _example()
    losses, r, load, params = m.train(steps=25, tokens=1000, experts=8, width=64, hidden=40)
    print("losses", [round(v, 4) for v in losses[::6]], flush=True)
    assert all(v == v for v in losses)
    assert losses[-1] < 0.8 * losses[0]
    assert int(load.sum()) == 1000 * 2
    row_ptr, col, val = m.shared_tokens(r)
    torch.cuda.synchronize()
    # The diagonal counts an expert's own tokens.
    E = 8
    rows = torch.repeat_interleave(torch.arange(E, device="cuda"), row_ptr.diff().long())
    diag = torch.zeros(E, device="cuda")
    on = rows == col
    diag[rows[on]] = val[on]
    assert torch.equal(diag, load)
    again = m.train(steps=25, tokens=1000, experts=8, width=64, hidden=40)[3]
    assert all(torch.equal(params[n], again[n]) for n in params), "two runs differ"
