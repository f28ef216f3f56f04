"""The inputs of step_hidden_reference tell two terms from one, and the right second term from
another row's, on the CPU: mistakes planted in the plain form leave its bound."""
import pytest

torch = pytest.importorskip("torch")
import expert_reference
import step_hidden_reference as ref

BF, HF = torch.bfloat16, torch.float16
SIZES = [(1, 4, 2, 32, 16), (3, 4, 2, 40, 65), (7, 5, 3, 33, 130)]


@pytest.mark.parametrize("dtype,unit", [(BF, 1.0), (HF, 1.0), (HF, 2.0 ** 11)])
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("T,E,k,D,F", SIZES)
def test_the_bound_needs_both_terms(T, E, k, D, F, eight, dtype, unit):
    t = ref.inputs(T, E, k, D, F, dtype, eight, T)
    col, val, _ = expert_reference.route((t[0].double() @ t[1].double().t()).float(), k)
    val = val.float()
    want, bound = ref.layer(t, col, val, unit)
    def outside(store):
        y = ref.layer(t, col, val, unit, store).to(dtype).double()
        return float(((y - want).abs() > bound).double().mean())
    assert outside(lambda h, i: ref.held(h, dtype, unit=unit)) == 0.0
    assert outside(lambda h, i: ref.held(h, dtype, 1)) > 0.2
    rest = {}
    def other_row(h, i):
        mine = ref.held(h, dtype, unit=unit) - h.to(dtype).double()
        rest[i] = mine
        return h.to(dtype).double() + rest.get(i - 1, mine.flip(0))
    assert outside(other_row) > 0.2


@pytest.mark.parametrize("eight", [False, True])
def test_small_values_of_float16_need_the_unit(eight):
    """Near 2^-9 a second term in steps of 2^-24 leaves 2^-16 of a value; in units of 2^-11 it keeps all of its bits."""
    t = ref.inputs(3, 4, 2, 40, 65, HF, eight, 5, size=2.0 ** -10)
    col, val, _ = expert_reference.route((t[0].double() @ t[1].double().t()).float(), 2)
    val = val.float()
    _, rough = ref.layer(t, col, val, 1.0)
    want, bound = ref.layer(t, col, val, 2.0 ** 11)
    y = ref.layer(t, col, val, 1.0, lambda h, i: ref.held(h, HF))
    assert bool(((y - want).abs() <= rough).all())
    y = ref.layer(t, col, val, 1.0, lambda h, i: ref.held(h, HF, unit=2.0 ** 11))
    assert bool(((y - want).abs() <= bound).all())


def test_large_scales_show_what_a_second_term_without_units_loses():
    t = list(ref.inputs(5, 6, 2, 264, 130, HF, True, 82, size=2.0 ** -12))
    t[5] = t[5] * 2.0 ** 12
    col, val, _ = expert_reference.route((t[0].double() @ t[1].double().t()).float(), 2)
    val = val.float()
    want, bound = ref.layer(t, col, val, 2.0 ** 11)
    y = ref.layer(t, col, val, 2.0 ** 11, lambda h, i: ref.held(h, HF)).to(HF).double()
    assert bool(((y - want).abs() > bound).any())   # one value outside fails a test
    y = ref.layer(t, col, val, 2.0 ** 11, lambda h, i: ref.held(h, HF, unit=2.0 ** 11)).to(HF).double()
    assert bool(((y - want).abs() <= bound).all())
