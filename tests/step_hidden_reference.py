"""Inputs on which the hidden vector's second term decides what expert_step returns, and the
64-bit result with a bound that only two terms meet.

x and w_in are small whole numbers and multiples of 2^-4, so that the sums of the first
product are exact.  A row of w_out has `TERMS` weights that are not 0, in pairs +w, -w of
neighbouring columns, whose hidden values differ by a few hundredths: y is a small
difference, and its own rounding hides nothing of theirs.

Bound of a hidden value h: 3 2^-20 |h| for exp, division and products in fp32, and what
holding it in two terms leaves.  The first term is off by at most u |h| (u = 2^-8 for bfloat16,
2^-11 for float16), the second by u of that; float16 also by half of its smallest step, 2^-25,
in the units that the second term is held in.  Sums add 2^-24 for each term of each
expert that is not 0, first and second, and as much again for the products."""
import torch

from expert_reference import EPS, FUN, TINY, U

TERMS = 8
E4 = torch.float8_e4m3fn


def inputs(T, E, k, D, F, dtype, eight, seed, size=1.0):
    """x, router, w_in, w_out, in_scale, out_scale on the CPU; h is about `size`, a power of two."""
    gen = torch.Generator().manual_seed(seed)
    def whole(lo, hi, *s):
        return torch.randint(lo, hi + 1, s, generator=gen).float()
    x = whole(-2, 2, T, D) * (torch.rand(T, D, generator=gen) < min(1.0, 32 / D))
    w_in = whole(-4, 4, E, 2 * F, D)
    up = w_in[:, F:]
    up[:, 1:F // 2 * 2:2] = up[:, 0:F // 2 * 2:2]
    at = torch.randint(0, D, (E, F // 2, 1), generator=gen)
    twin = up[:, 1:F // 2 * 2:2]
    twin.scatter_(2, at, -twin.gather(2, at) + 1.0)
    w_in[:, 1:F // 2 * 2:2] = w_in[:, 0:F // 2 * 2:2]
    w_out = torch.zeros(E, D, F)
    pairs = min(TERMS // 2, F // 2)
    for d in range(D):
        which = torch.randint(0, F // 2, (E, pairs), generator=gen)
        w = whole(1, 7, E, pairs)
        w_out[:, d].scatter_(1, 2 * which, w)
        w_out[:, d].scatter_(1, 2 * which + 1, -w)
    router = torch.randn(E, D, generator=gen)
    if not eight:
        w_in[:, :F] /= 16.0
        w_in[:, F:] *= size / 16.0
        return x.to(dtype), router, w_in.to(dtype), w_out.to(dtype), None, None
    up128 = lambda n: -(-n // 128)
    # The scales of blocks that hold gate rows and up rows are one: size is then on both.
    s_in = torch.full((E, up128(2 * F), up128(D)), size ** 0.5 / 16.0)
    return x.to(dtype), router, w_in.to(E4), w_out.to(E4), s_in, torch.ones(E, up128(D), up128(F))


def spread(w, scale):
    if scale is None:
        return w.double()
    rows, cols = w.shape[1:]
    return w.double() * scale.double().repeat_interleave(128, 1)[:, :rows].repeat_interleave(128, 2)[:, :, :cols]


def held(h, dtype, terms=2, unit=1.0):
    """h (fp32) as `terms` values of dtype, the second times `unit`: their sum in 64 bits."""
    first = h.to(dtype)
    out = first.double()
    if terms == 2:
        out = out + ((h - first.float()) * unit).to(dtype).double() / unit
    return out


def layer(t, col, val, unit, store=None):
    """(y, bound) of the layer for the routing (col, val), with the second term in units of 1 / `unit`; with `store`
    the value from hidden values of fp32 that it changes, and no bound."""
    x, _, w_in, w_out, in_scale, out_scale = t
    dtype = x.dtype
    u = U[dtype]
    floor = (2.0 ** -25 if dtype is torch.float16 else TINY[dtype]) / unit
    x, w_in, w_out = x.double(), spread(w_in, in_scale), spread(w_out, out_scale)
    (T, D), F, k = x.shape, w_out.shape[2], col.shape[1]
    y, b, m = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    for i in range(k):
        for r in range(T):
            e = int(col[r, i])
            if e < 0:
                continue
            g, up = (w_in[e] @ x[r]).split(F)
            h = g * torch.sigmoid(g) * up
            w = float(val[r, i])
            if store is not None:
                y[r] += w * (w_out[e] @ store(h.float(), r * k + i))
                continue
            dh = 3 * FUN * h.abs()
            err = dh + u * u * (h.abs() + dh) + floor
            y[r] += w * (w_out[e] @ h)
            b[r] += abs(w) * (w_out[e].abs() @ err)
            m[r] += abs(w) * (w_out[e].abs() @ (h.abs() + err))
    if store is not None:
        return y
    b = b + 4 * k * TERMS * EPS * m
    return y, b + u * (y.abs() + b) + TINY[dtype]
