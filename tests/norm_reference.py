"""Layer norm and its gradient in 64 bits, on the CPU, with bounds on what fp32 sums
and one rounding of a value to its type can add.

Bounds, to first order with room for the second: a sum of a row's D terms has at
most 64 additions one after the other, so it is off by 64 2^-24 of the terms' magnitudes;
sums over T rows by T + 64 of them; every other operation by 2^-24, the square root and
the division by 2^-23."""
import torch

from expert_reference import EPS

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -126}
ROW = 64 * EPS


def rounded(v, b, dtype):
    # A value whose range reaches past the type's largest is rounded to an infinity, rightly: with one column n is
    # 0, but kept in 8 bits it is (x^ - x) / sqrt(eps), and dx = -r n^2 dy leaves float16.
    most = torch.finfo(dtype).max
    return v, torch.where(v.abs() + b < most, b + U[dtype] * (v.abs() + b) + TINY[dtype], torch.inf)


def layer_norm(x, weight, bias, eps, grad=None, at=None):
    """{name: (value, bound)}; `at`: the rows that the gradients are taken at, where not x."""
    t, tw = x.dtype, weight.dtype
    x, w = x.double(), weight.double()
    T, D = x.shape
    eps = float(torch.tensor(eps, dtype=torch.float32))

    def mean(v):
        return v.mean(1, keepdim=True)

    m = mean(x)
    dm = ROW * mean(x.abs()) + 2 * EPS * m.abs()
    d = x - m
    v = mean(d * d)
    dd = dm + EPS * (d.abs() + dm)
    dv = mean(2 * d.abs() * dd + dd * dd) + (ROW + 4 * EPS) * mean((d.abs() + dd) ** 2)
    part = (dv + 2 * EPS * (v + eps)) / (v + eps)   # relative, of v + eps
    r = 1.0 / torch.sqrt(v + eps)
    # |(1 - p)^(-1/2) - 1| <= p below 1/2: beyond it nothing is promised.
    dr = torch.where(part < 0.5, r * (part + 6 * EPS), torch.inf)

    def unit(x):
        d = x - m
        dd = dm + EPS * (d.abs() + dm)
        n = d * r
        return n, 1.01 * (dd * (r + dr) + d.abs() * dr) + 3 * EPS * n.abs()

    n, dn = unit(x)
    b = torch.zeros(D, dtype=torch.float64) if bias is None else bias.double()
    out = {"y": rounded(n * w + b, w.abs() * dn + 4 * EPS * ((n * w).abs() + b.abs()), t)}
    if grad is None:
        return out
    if at is not None:
        n, dn = unit(at.double())
    dy = grad.double()
    a = dy * w
    s1, s2 = mean(a), mean(a * n)
    ds1 = (ROW + 3 * EPS) * mean(a.abs())
    ds2 = mean(a.abs() * dn) + (ROW + 5 * EPS) * mean(a.abs() * (n.abs() + dn))
    dx = r * (a - s1 - n * s2)
    size = a.abs() + s1.abs() + (n * s2).abs()
    ex = 1.01 * ((r + dr) * (ds1 + (n.abs() + dn) * ds2 + s2.abs() * dn + 8 * EPS * size) + dr * size)
    out["grad_x"] = rounded(dx, ex, t)
    k = (T + 64) * EPS
    p = dy.abs() * (n.abs() + dn)
    out["grad_weight"] = rounded((dy * n).sum(0), (dy.abs() * dn).sum(0) + k * p.sum(0), tw)
    out["grad_bias"] = rounded(dy.sum(0), k * dy.abs().sum(0), tw)
    return out
