"""The global gradient norm and its clipping, against sums in 64 bits.

The squares are summed in fp64: the norm is within an fp32 rounding, 2^-24, of
the exact one (2^-23 allowed for the last place of the sums); a scaled element
is off by the factor's rounding and its own product's, 2 2^-24, and by one
rounding to its type."""
import math

import pytest

torch = pytest.importorskip("torch")
sg = pytest.importorskip("spgemm_symbolic_row_amd")

pytestmark = pytest.mark.gpu

F32, BF, HF = torch.float32, torch.bfloat16, torch.float16
HALF_ULP = {F32: 2.0 ** -24, BF: 2.0 ** -8, HF: 2.0 ** -11}
TINY = {F32: 2.0 ** -149, BF: 2.0 ** -133, HF: 2.0 ** -25}


def check(grads, max_norm, outs=None):
    norm64 = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    c = min(1.0, max_norm / (norm64 + 1e-6))
    want = [g.double() * c for g in grads]
    target = grads if outs is None else outs
    norm = sg.clip_grad_norm(grads, max_norm, out=outs)
    torch.cuda.synchronize()
    assert norm.dtype == F32 and norm.shape == ()
    assert abs(float(norm) - norm64) <= 2.0 ** -23 * norm64
    for i, (o, w) in enumerate(zip(target, want)):
        bound = (HALF_ULP[o.dtype] + 3 * 2.0 ** -24) * w.abs() + TINY[o.dtype]
        err = (o.double() - w).abs()
        assert bool((err <= bound).all()), f"tensor {i}: {float((err / bound).max())} of its bound"


def randn(n, dtype, seed, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, generator=gen, device="cuda") * scale).to(dtype)


@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("sizes", [[1], [5, 0, 7], [16384], [16385, 3, 100000], list(range(1, 230))])
def test_clip(dtype, sizes):
    print(f"clip {dtype}, {len(sizes)} tensors, {sum(sizes)} elements", flush=True)
    for max_norm in (0.25, 1e9, 0.0):
        check([randn(n, dtype, i) for i, n in enumerate(sizes)], max_norm)


def test_mixed_types_into_other_types():
    kinds = [F32, BF, HF]
    grads = [randn(1000 + i, kinds[i % 3], i, 0.1) for i in range(12)]
    outs = [torch.empty(g.shape, dtype=kinds[(i // 3) % 3], device="cuda") for i, g in enumerate(grads)]
    check(grads, 0.5, outs)


def test_offsets_that_break_alignment():
    for dtype in (F32, BF):
        base = randn(5000, dtype, 1)
        for a, b in ((1, 0), (0, 1), (3, 3), (8, 4)):
            g = base[a:a + 3001]
            o = torch.full((4000,), float("nan"), dtype=dtype, device="cuda")
            check([g], 0.3, [o[b:b + 3001]])
            assert bool(torch.isnan(o[:b]).all()) and bool(torch.isnan(o[b + 3001:]).all())


def test_more_work_than_partial_sums():
    n = 2100 * 16384 + 11
    check([randn(n, BF, 0, 0.01), randn(777, F32, 1), randn(3, HF, 2)], 1.0)


def test_extremes():
    big = torch.full((1000,), 3e38, device="cuda")   # squares beyond fp32
    out = torch.empty_like(big)
    check([big / 100], 1.0, [out])
    assert bool(torch.isinf(sg.clip_grad_norm([big.clone()], 1.0))) is False or \
        float(big.double().square().sum().sqrt()) > 3.4e38
    small = torch.full((1000,), 1e-30, device="cuda")
    check([small], 1e-31)
    check([torch.zeros(10, device="cuda")], 1.0)
    for bad in (float("nan"), float("inf")):
        g = torch.ones(100, device="cuda")
        g[7] = bad
        n = sg.clip_grad_norm([g], 1.0)
        torch.cuda.synchronize()
        assert (math.isnan if math.isnan(bad) else math.isinf)(float(n))
        assert math.isnan(float(g[7]))
        rest = torch.cat([g[:7], g[8:]])
        assert bool(torch.isnan(rest).all() if math.isnan(bad) else (rest == 0).all())


def test_same_bits_twice():
    grads = [randn(100003, F32, 1), randn(50001, BF, 2)]
    outs = [[torch.empty_like(g) for g in grads] for _ in range(2)]
    n = [sg.clip_grad_norm(grads, 0.1, out=o) for o in outs]
    torch.cuda.synchronize()
    assert torch.equal(n[0], n[1]) and all(torch.equal(a, b) for a, b in zip(*outs))


def test_refusals():
    g = torch.ones(4, device="cuda")
    for args in (([],), ([g.cpu()],), ([g.double()],), ([torch.ones(4, 4, device="cuda").t()],)):
        with pytest.raises((TypeError, ValueError)):
            sg.clip_grad_norm(*args, 1.0)
    with pytest.raises(ValueError):
        sg.clip_grad_norm([g], 1.0, out=[])
    with pytest.raises(ValueError):
        sg.clip_grad_norm([g], 1.0, out=[torch.ones(5, device="cuda")])
    for m in (-1.0, float("nan")):
        with pytest.raises(sg.SpgemmError) as e:
            sg.clip_grad_norm([g], m)
        assert e.value.status == -1
    torch.cuda.synchronize()
    assert bool((g == 1).all())


def test_a_norm_beyond_fp32():
    """The norm is infinite in fp32, the factor below its normal numbers; the elements are right."""
    for dtype, size, n in ((F32, 3e38, 1000), (BF, 3e38, 5003), (F32, 1e36, 40_000_000)):
        g = torch.full((n,), size, device="cuda").to(dtype)
        norm64 = float(g[0]) * math.sqrt(n)
        for max_norm in (1.0, 1e-3):
            out = torch.empty(n, device="cuda")
            norm = sg.clip_grad_norm([g], max_norm, out=[out])
            torch.cuda.synchronize()
            assert math.isinf(float(norm)) == (norm64 > 3.4028235e38)
            want = float(g[0]) * (max_norm / norm64)
            off = float(((out.double() - want).abs() / want).max())
            assert off <= 4 * 2.0 ** -24, (dtype, size, max_norm)
