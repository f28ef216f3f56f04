"""Plain 64-bit forms of the expert-layer operators, on the CPU, with bounds on
what fp32 sums and one rounding of a value to the tensors' type can add.

Bounds: an fp32 sum of K products is off by at most 2 K 2^-24 times the sum of
their magnitudes; exp and the divisions of a sigmoid by at most 2^-20
relative; a rounding by u |v| (half a unit in the last of 8 or 11 bits: 2^-8 for bfloat16, 2^-11 for float16) or,
where float16 is subnormal, 2^-25."""
import torch

EPS = 2.0 ** -24
FUN = 2.0 ** -20
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}


def route(logits, k, scores="softmax", bias=None, groups=1, top_groups=0, renormalise=True,
          scale=1.0, active=None, grad=None):
    """(col, val, grad_logits) row by row; keys in fp32 as the operator's definition says."""
    T, E = logits.shape
    z32 = logits.float()
    key = z32 if scores == "softmax" else 1.0 / (1.0 + torch.exp(-z32))
    if bias is not None:
        key = key + bias
    col = torch.full((T, k), -1, dtype=torch.int32)
    val = torch.zeros(T, k, dtype=torch.float64)
    dz = torch.zeros(T, E, dtype=torch.float64)
    per = E // groups
    for t in range(T):
        z = z32[t].double()
        live = [e for e in range(E) if z32[t, e] > -torch.inf and key[t, e] > -torch.inf
                and (active is None or bool(active[t]))]
        allowed = live
        if groups > 1 and top_groups:
            score = {}
            for g in range(groups):
                ks = sorted((key[t, e] for e in live if e // per == g), reverse=True)
                if ks:
                    score[g] = ks[0] + ks[1] if scores == "sigmoid" and len(ks) > 1 else ks[0]
            best = sorted(score, key=lambda g: (-float(score[g]), g))[:top_groups]
            allowed = [e for e in live if e // per in best]
        pick = sorted(sorted(allowed, key=lambda e: (-float(key[t, e]), e))[:k])
        if not pick:
            continue
        among = pick if renormalise or scores == "sigmoid" else live
        if scores == "softmax":
            p = torch.zeros(E, dtype=torch.float64)
            p[among] = torch.softmax(z[among], 0)
            w = p[pick]
        else:
            p = torch.sigmoid(z)
            total = p[pick].sum() + 1e-20 if renormalise else 1.0
            w = p[pick] / total
        col[t, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
        val[t, :len(pick)] = w * scale
        if grad is not None:
            dw = torch.zeros(E, dtype=torch.float64)
            dw[pick] = grad[t, :len(pick)].double() * scale
            if scores == "softmax":
                dz[t] = p * (dw - (p * dw).sum())
            else:
                d = dw[pick]
                if renormalise:
                    d = (d - (w * d).sum()) / total
                dz[t, pick] = d * p[pick] * (1 - p[pick])
    return col, val, dz


def experts(x, w_in, w_out, col, val, grad_y=None):
    """{name: (value, bound)} of y and, with grad_y, of the gradients."""
    t16 = x.dtype
    u16, tiny = U[t16], TINY[t16]
    x, w_in, w_out, val = x.double(), w_in.double(), w_out.double(), val.double()
    (T, D), (E, _, F), k = x.shape, w_out.shape, col.shape[1]
    zero = torch.zeros_like
    y, yb, ym = zero(x), zero(x), zero(x)
    gx, gxb = zero(x), zero(x)
    gi, gib, go, gob = zero(w_in), zero(w_in), zero(w_out), zero(w_out)
    gv, gvb = zero(val), zero(val)
    dy = None if grad_y is None else grad_y.double()
    for e in range(E):
        t, i = torch.nonzero(col == e, as_tuple=True)
        if not len(t):
            continue
        xe, w = x[t], val[t, i][:, None]
        a, w2 = w_in[e], w_out[e]
        pre, mag = xe @ a.T, xe.abs() @ a.abs().T
        g, u, dG, dU = pre[:, :F], pre[:, F:], 2 * D * EPS * mag[:, :F], 2 * D * EPS * mag[:, F:]
        s = torch.sigmoid(g)
        silu, slope = g * s, s * (1 + g * (1 - s))
        h = silu * u
        dh_ = 1.1 * dG * u.abs() + (silu.abs() + 1.1 * dG) * dU + 3 * FUN * h.abs()   # fp32 error of h
        hr = dh_ + u16 * (h.abs() + dh_) + tiny                                       # and as stored
        y.index_add_(0, t, w * (h @ w2.T))
        yb.index_add_(0, t, w.abs() * ((hr + 2 * F * EPS * (h.abs() + hr)) @ w2.abs().T))
        ym.index_add_(0, t, w.abs() * (h.abs() @ w2.abs().T))
        if dy is None:
            continue
        d = dy[t]
        q, dq = d @ w2, 2 * D * EPS * (d.abs() @ w2.abs())
        gv[t, i] = (h * q).sum(1)
        gvb[t, i] = (h.abs() * dq + dh_ * (q.abs() + dq)
                     + 2 * (F + 64) * EPS * (h * q).abs()).sum(1)
        dg, du = w * q * u * slope, w * q * silu
        aw = w.abs()
        eg = aw * (dq * (u.abs() + dU) * (slope.abs() + dG) + q.abs() * dU * (slope.abs() + dG)
                   + q.abs() * u.abs() * 0.6 * dG) + 6 * FUN * aw * (q * u).abs() * (1 + g.abs())
        eu = aw * (dq * (silu.abs() + 1.1 * dG) + q.abs() * 1.1 * dG) + 6 * FUN * du.abs()
        dgu = torch.cat([dg, du], 1)
        err = torch.cat([eg, eu], 1)
        err = err + u16 * (dgu.abs() + err) + tiny
        gx.index_add_(0, t, dgu @ a)
        gxb.index_add_(0, t, (err + 4 * F * EPS * dgu.abs()) @ a.abs())
        n = len(t)
        gi[e] = dgu.T @ xe
        gib[e] = (err + 2 * n * EPS * dgu.abs()).T @ xe.abs()
        hw = aw * h.abs()
        hwe = aw * dh_ + FUN * hw
        hwe = hwe + u16 * (hw + hwe) + tiny
        go[e] = d.T @ (w * h)
        gob[e] = d.abs().T @ (hwe + 2 * n * EPS * hw)
    def rounded(v, b):
        return v, b + u16 * (v.abs() + b) + tiny
    out = {"y": rounded(y, yb + 2 * k * EPS * ym)}
    if dy is not None:
        out |= {"grad_x": rounded(gx, gxb * (1 + 4 * k * EPS) + 4 * k * EPS * gx.abs()),
                "grad_w_in": rounded(gi, gib), "grad_w_out": rounded(go, gob),
                "grad_val": (gv, gvb + 1e-30)}
    return out


def assert_within(got, value, bound, what):
    err = (got.double().cpu() - value).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} outside; first {torch.nonzero(bad)[0].tolist()}: "
        f"{got.double().cpu()[bad][0].item()} for {value[bad][0].item()}, bound {bound[bad][0].item()}")
    if err.numel():
        print(f"{what}: {err.numel()} values, largest error {float((err / bound).max()):.3g} of the "
              "bound", flush=True)
