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


def beyond(dtype, eight, fp32):
    """One token whose hidden value is beyond the type in every column, in fp32 too or just not, and one of others."""
    E, D, F = 2, 32, 40
    w_in, w_out = torch.zeros(E, 2 * F, D), torch.ones(E, D, F)
    x = torch.ones(2, D)
    w_out[:, 1::2] = -1.0
    if dtype is HF:
        w_in[0] = 12.0                             # h = 384 * 384
    else:
        # 2^128 (1 - 2^-9), half way between bfloat16's largest value and what would follow; or 2^130.
        w_in[0] = 2.0 ** 59
        w_in[0, F:, 16:] *= 1.0 - 2.0 ** -8
        if fp32:
            w_in[0] *= 2.0
    w_in[1] = 2.0 ** -6
    router = torch.zeros(E, D)
    router[0, 0], router[1, 0] = 1.0, -1.0
    x[1, 0] = -1.0
    if not eight:
        return [v.cuda() for v in (x.to(dtype), router, w_in.to(dtype), w_out.to(dtype))], {}
    codes = torch.full((E, 2 * F, D), 1.0)
    scale = torch.ones(E, 1, 1)
    scale[0], scale[1] = w_in[0].max(), 2.0 ** -6   # one block: h = 2^128 or more for bfloat16
    return ([v.cuda() for v in (x.to(dtype), router, codes.to(ref.E4), w_out.to(ref.E4))],
            dict(in_scale=scale.cuda(), out_scale=torch.ones(E, 1, 1).cuda()))


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("dtype,fp32", [(BF, False), (BF, True), (HF, False)])
def test_a_hidden_value_beyond_its_type_is_infinite(dtype, fp32, eight):
    """As it is in `experts`, and not NaN."""
    print(dtype, fp32, eight, flush=True)
    args, how = beyond(dtype, eight, fp32)
    y, r = sg.expert_step(*args, 1, **how)
    torch.cuda.synchronize()
    assert r.col.tolist() == [[0], [1]]
    sign = torch.ones(32, device="cuda")
    sign[1::2] = -1.0
    assert torch.equal(y[0].float(), sign * float("inf"))
    if not eight:
        z = sg.experts(args[0], args[2], args[3], r.col, r.val)
        assert torch.equal(y[0], z[0])
    # g = u = 30 / 64 in every column, which sum to 40 h.
    g = torch.tensor(30 / 64, dtype=torch.float64)
    h = float(g * torch.sigmoid(g) * g) * 40
    u = {BF: 2.0 ** -8, HF: 2.0 ** -11}[dtype]
    assert bool(((y[1].double() - sign.double() * h).abs() <= (u + 2.0 ** -14) * h).all())


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -6, 2.0 ** -10])
@pytest.mark.parametrize("T,E,k,D,F", SIZES)
def test_float16_holds_small_values_in_both_terms(T, E, k, D, F, size, eight):
    """The second term is held in units of 2^-11, so that what it leaves does not grow beside small values."""
    check(T, E, k, D, F, HF, eight, 2.0 ** 11, size=size)


@pytest.mark.parametrize("T,k", [(1, 2), (5, 2), (16, 3)])
def test_small_values_of_float16_with_large_scales(T, k):
    """Hidden values near 2^-12 that the scales of 8-bit weights bring back into y's range: the steps of an unscaled
    second term would be 2^-13 of them and more."""
    E, D, F = 6, 264, 130
    t = list(ref.inputs(T, E, k, D, F, HF, True, 77 + T, size=2.0 ** -12))
    t[5] = t[5] * 2.0 ** 12
    g = [v.cuda() for v in t]
    y, r = sg.expert_step(*g[:4], k, in_scale=g[4], out_scale=g[5])
    torch.cuda.synchronize()
    assert_within(y, *ref.layer(t, r.col.cpu(), r.val.cpu(), 2.0 ** 11), "y")
