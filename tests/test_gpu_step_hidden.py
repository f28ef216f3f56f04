"""expert_step's hidden vector in two terms, on inputs whose results one term, or another row's
second term, would change (test_step_hidden_cpu plants both)."""
import pytest

torch = pytest.importorskip("torch")
sg = pytest.importorskip("spgemm_symbolic_row_amd")
import step_hidden_reference as ref
from expert_reference import assert_within

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16

SIZES = [
    # T, E, k, D, F: one and two products a step, one to sixteen parts of K, ends of K, rows of x that stay in memory
    (1, 4, 2, 32, 16),
    (1, 8, 8, 256, 200),
    (2, 3, 1, 17, 31),
    (3, 4, 2, 40, 65),
    (4, 24, 3, 2048, 64),
    (7, 12, 4, 520, 130),
    (8, 6, 2, 100, 384),
    (13, 20, 4, 264, 96),
    (16, 40, 6, 512, 72),
    (16, 300, 10, 72, 33),
    (16, 4, 2, 4160, 48),
]


def check(T, E, k, D, F, dtype, eight, unit, **how):
    print(f"T={T} E={E} k={k} D={D} F={F} {dtype} {'e4m3' if eight else '16-bit'} {how}", flush=True)
    t = ref.inputs(T, E, k, D, F, dtype, eight, T + D, **how)
    g = [None if v is None else v.cuda() for v in t]
    y, r = sg.expert_step(*g[:4], k, in_scale=g[4], out_scale=g[5])
    torch.cuda.synchronize()
    assert bool((r.col >= 0).all())
    assert_within(y, *ref.layer(t, r.col.cpu(), r.val.cpu(), unit), "y")


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,E,k,D,F", SIZES)
def test_both_terms(T, E, k, D, F, dtype, eight):
    check(T, E, k, D, F, dtype, eight, 1.0)
