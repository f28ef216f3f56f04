"""Rows kept in 8 bits, on the CPU, from the definition: every code's value is listed and the
nearest one is looked up."""
import torch

E4M3 = torch.tensor([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7)
                     for e in range(16) for m in range(8)][:127], dtype=torch.float64)


def nearest_e4m3(a, most):
    """The nearest code value of a >= 0 that is not above `most`; of two the one with an even code."""
    hi = torch.searchsorted(E4M3, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = E4M3[hi] - a, a - E4M3[lo]
    at = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.minimum(E4M3[at], most)


def kept(x):
    """What the 8 bits of x's rows (T x D) stand for, in 64 bits."""
    half = x.dtype == torch.float16
    out = torch.empty(x.shape, dtype=torch.float64)
    for c in range(0, x.shape[1], 128):
        v = x[:, c:c + 128].double()
        finite = torch.isfinite(v)
        most = torch.where(finite, v.abs(), 0.0).amax(1, keepdim=True)
        s = torch.full_like(most, 2.0 ** (-15 if half else -117))
        while bool((most > 448 * s).any()):
            s = torch.where(most > 448 * s, 2 * s, s)
        top = torch.where(s == 2.0 ** (8 if half else 120), 240.0, 448.0).to(torch.float64)
        a = torch.where(finite, v.abs(), 0.0) / s
        q = nearest_e4m3(a, top.expand_as(a)) * s * torch.sign(v)
        out[:, c:c + 128] = torch.where(finite, q, torch.nan)
    return out
