"""float64 oracle of the gated linear recurrence and of the group norm, with error bounds.

Test infrastructure only: the definitions token by token (recurrence) and row by
row (norm) in torch float64 on the CPU, sharing no code with the GPU path.  Next
to each value stands a bound on the error of a float32 evaluation of the same
formula.  With U = 2^-24 (half a step of float32, relative) the bounds count

  exp(g):        (2 |g| + 4) U relative: the product g log2(e) is rounded (|g| U,
                 and half that again for the constant), the base-2 exponential is
                 good to one step (2 U), one U to spare.  It has no subnormal results: a
                 value below 2^-126 comes out as 0, an absolute error below 2^-126,
                 which is 2^-126 / a relative;
  1 - exp(g):    (|g| + 8) U relative: a polynomial of eight rounded steps for small
                 |g|; elsewhere the exponential's error and one rounding of the
                 difference, over a value of at least 0.39;
  h = a h' + u:  the error of h' times a, |a h'| times that of a, |u| times that of u
                 (and of its product), one rounding of the sum.  The bound follows the
                 same recurrence in absolute values.  A kernel that joins blocks
                 of rows by their products of decays, exp of a sum of g, makes per
                 block the error of that sum (at most 64 U sum |g|) and of one exp,
                 in place of those of the rows' exponentials; twice the row-by-row
                 bound covers both (the sum's error counts when |g| is large, where
                 the decayed value it scales is correspondingly small: its part is
                 a |h'| 64 U |g| per row, added below).
"""
import torch

U = 2.0 ** -24
F64 = torch.float64


def half_step(dtype):
    """Half a rounding step of a type, relative."""
    return torch.finfo(dtype).eps / 2


def rounded(value, bound, dtype):
    """Bound on the distance of a stored result from `value` when it was off by `bound` before rounding."""
    tiny = torch.finfo(dtype).tiny * torch.finfo(dtype).eps  # a subnormal step
    return bound + (value.abs() + bound) * half_step(dtype) + tiny


def _terms(x, g, complement):
    a = g.exp()
    ea = (2 * g.abs() + 4) * U
    ea = torch.where(a == 0, torch.zeros_like(ea), ea + 2.0 ** -126 / a)  # exp(-inf) is exact
    if not complement:
        return a, ea, x, torch.zeros_like(x)
    m = -torch.expm1(g)
    em = torch.where(a == 0, torch.zeros_like(g), (g.abs() + 8) * U)
    return a, ea, m * x, (m * x).abs() * (em + U)


def _join(g, a):
    """What the joining of blocks adds, relative to a |h'|: the rounding of the sum of g."""
    return torch.where(a == 0, torch.zeros_like(g), 64 * U * g.abs())


def scan(x, g, cu, s0=None, complement=False):
    """o, final [N, D], before (h_{t-1} of every row), and bounds of o/final (float64 CPU tensors).
    Rows outside the sequences hold zeros."""
    x, g = x.detach().cpu().to(F64), g.detach().cpu().to(F64)
    T, D = x.shape
    edges = [int(c) for c in cu]
    N = len(edges) - 1
    a, ea, u, eu = _terms(x, g, complement)
    ea = ea + _join(g, a)
    o, ob, before, bb = (torch.zeros(T, D, dtype=F64) for _ in range(4))
    fs, fb = torch.zeros(N, D, dtype=F64), torch.zeros(N, D, dtype=F64)
    for i in range(N):
        h = torch.zeros(D, dtype=F64) if s0 is None else s0[i].detach().cpu().to(F64)
        b = torch.zeros(D, dtype=F64)
        for t in range(edges[i], edges[i + 1]):
            before[t], bb[t] = h, b
            carried = torch.where(a[t] == 0, torch.zeros_like(h), a[t] * h)
            b = torch.where(a[t] == 0, torch.zeros_like(b), a[t] * b) + carried.abs() * ea[t] + eu[t]
            h = carried + u[t]
            b = b + h.abs() * U
            o[t], ob[t] = h, b
        fs[i], fb[i] = h, b
    return {"o": o, "o_bound": 2 * ob, "final": fs, "final_bound": 2 * fb, "before": before, "before_bound": 2 * bb}


def scan_backward(x, g, cu, d_o, d_final=None, s0=None, complement=False):
    """Gradients dx, dg, ds0 and their bounds (float32 evaluation, before the rounding of the stores)."""
    f = scan(x, g, cu, s0, complement)
    x, g, d_o = (t.detach().cpu().to(F64) for t in (x, g, d_o))
    T, D = x.shape
    edges = [int(c) for c in cu]
    N = len(edges) - 1
    a, ea, _, _ = _terms(x, g, complement)
    ej = ea + _join(g, a)
    m = -torch.expm1(g)
    em = torch.where(a == 0, torch.zeros_like(g), (g.abs() + 8) * U)
    dx, dxb, dg, dgb = (torch.zeros(T, D, dtype=F64) for _ in range(4))
    ds0, ds0b = torch.zeros(N, D, dtype=F64), torch.zeros(N, D, dtype=F64)
    for i in range(N):
        e = torch.zeros(D, dtype=F64) if d_final is None else d_final[i].detach().cpu().to(F64)
        b = torch.zeros(D, dtype=F64)
        for t in range(edges[i + 1] - 1, edges[i] - 1, -1):
            e = e + d_o[t]
            b = b + e.abs() * U
            p, pb = f["before"][t], f["before_bound"][t]
            if complement:
                p = p - x[t]
                pb = pb + p.abs() * U
                # 1 - a may be kept in place of a: a is then off by the error of 1 - a and a rounding
                dx[t], dxb[t] = m[t] * e, m[t].abs() * (2 * b + e.abs() * (em[t] + U))
                slack = (em[t] + U) * m[t]
            else:
                dx[t], dxb[t] = e, 2 * b
                slack = torch.zeros(D, dtype=F64)
            dg[t] = e * a[t] * p
            dgb[t] = a[t] * (2 * b * p.abs() + e.abs() * pb + 2 * b * pb) + dg[t].abs() * (ea[t] + 3 * U)
            b = a[t] * b + (a[t] * e).abs() * (ej[t] + U) + slack * e.abs()
            e = a[t] * e
        ds0[i], ds0b[i] = e, 2 * b
    return {"dx": dx, "dx_bound": dxb, "dg": dg, "dg_bound": dgb, "ds0": ds0, "ds0_bound": ds0b}


def decode(x, g, cache, slots, complement=False):
    """One token per entry: o, the new cache and their bounds."""
    x, g = x.detach().cpu().to(F64), g.detach().cpu().to(F64)
    new = cache.detach().cpu().to(F64).clone()
    a, ea, u, eu = _terms(x, g, complement)
    o, ob, cb = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(new)
    for i, s in enumerate(int(s) for s in slots):
        if 0 <= s < new.shape[0]:
            carried = torch.where(a[i] == 0, torch.zeros_like(a[i]), a[i] * new[s])
            b = carried.abs() * ea[i] + eu[i]
            new[s] = carried + u[i]
            cb[s] = b + new[s].abs() * U
            o[i], ob[i] = new[s], cb[s]
    return {"o": o, "o_bound": ob, "cache": new, "cache_bound": cb}


# ------------------------------------------------------------------- norm

def _activation(name, v):
    """act(v), act'(v) and bounds of their float32 evaluations.  exp(-v) is off by (2 |v| + 4) U relative,
    the sum and the quotient add 3 U, so s by (2 |v| + 8) U absolute at most (s (1 - s) <= 1/4 scales the
    exponential's part), and by 2^-126 more: exp(-v) past 2^126 makes s a subnormal or, past 2^128, 0.
    s v and s (1 + v (1 - s)) carry that on with the factors they multiply it by."""
    if name in (None, "none"):
        return v, torch.ones_like(v), torch.zeros_like(v), torch.zeros_like(v)
    s = torch.sigmoid(v)
    es = s * (1 - s) * (2 * v.abs() + 4) * U + s * 4 * U + 2.0 ** -126
    if name == "sigmoid":
        return s, s * (1 - s), es, es * (1 + 2 * s) + s * (1 - s) * 2 * U + s * U
    f, df = v * s, s * (1 + v * (1 - s))
    ef = v.abs() * es + f.abs() * U
    edf = es * (1 + v.abs()) * 2 + s * (1 + 2 * v.abs()) * 4 * U
    return f, df, ef, edf


def norm(x, weight=None, bias=None, gate=None, activation=None, subtract_mean=True, eps=1e-5, d_y=None):
    """y (and with d_y the gradients dx, dgate, dweight, dbias) of the group norm over the last dimension
    of x [T, G, V], with bounds.  A sum of V values in float32, at most 64 of them one after another and
    the rest pairwise, is off by at most S = 80 U times the sum of the absolute values."""
    x = x.detach().cpu().to(F64)
    T, G, V = x.shape
    one = torch.ones(G, V, dtype=F64)
    w = one if weight is None else weight.detach().cpu().to(F64).expand(G, V)
    b = 0 * one if bias is None else bias.detach().cpu().to(F64).expand(G, V)
    S = 80 * U
    mean = x.mean(-1, keepdim=True) if subtract_mean else torch.zeros(T, G, 1, dtype=F64)
    em = (x.abs().mean(-1, keepdim=True) * S + mean.abs() * U) if subtract_mean else torch.zeros_like(mean)
    d = x - mean
    ed = em + d.abs() * U
    var = (d * d).mean(-1, keepdim=True)
    # the squares of values off by ed, their sum, eps
    ev = (2 * d.abs() * ed + ed * ed).mean(-1, keepdim=True) + var * (S + 2 * U)
    rstd = (var + eps) ** -0.5
    er = 0.5 * ev / (var + eps) + 4 * U  # relative
    xhat = d * rstd
    ex = ed * rstd + xhat.abs() * (er + U)
    n = xhat * w + b
    en = ex * w.abs() + n.abs() * U + (xhat * w).abs() * U
    z = None if gate is None else gate.detach().cpu().to(F64)
    f, df, ef, edf = _activation(activation, n if z is None else z)
    if z is None:
        slope = 1.1 if activation == "silu" else 1.0
        y, ey = f, ef + en * slope
    else:
        y, ey = n * f, n.abs() * ef + f.abs() * en + (n * f).abs() * U
    res = {"y": y, "y_bound": ey}
    if d_y is None:
        return res
    dy = d_y.detach().cpu().to(F64)
    if z is None:
        dn = dy * df
        edn = dy.abs() * (edf + en * 0.6) + dn.abs() * U  # |act''| <= 1/2 for silu, below 0.1 for sigmoid
    else:
        dn = dy * f
        edn = dy.abs() * ef + dn.abs() * U
        res["dgate"] = dy * n * df
        res["dgate_bound"] = dy.abs() * (n.abs() * edf + en * df.abs()) + res["dgate"].abs() * 3 * U
    q = dn * w
    eq = edn * w.abs() + q.abs() * U
    s1 = q.mean(-1, keepdim=True) if subtract_mean else torch.zeros_like(mean)
    es1 = (eq.mean(-1, keepdim=True) + q.abs().mean(-1, keepdim=True) * S) if subtract_mean else torch.zeros_like(mean)
    s2 = (q * xhat).mean(-1, keepdim=True)
    es2 = (eq * xhat.abs() + q.abs() * ex).mean(-1, keepdim=True) + (q * xhat).abs().mean(-1, keepdim=True) * (S + U)
    r = q - s1 - xhat * s2
    er2 = eq + es1 + xhat.abs() * es2 + ex * s2.abs() + (q.abs() + s1.abs() + 2 * (xhat * s2).abs()) * 2 * U
    res["dx"], res["dx_bound"] = r * rstd, er2 * rstd + (r * rstd).abs() * (er + U)
    # sums over the tokens (and groups): at most rows / 64 + 64 values one after another in any partial sum
    for name, p, term, eterm in (("dweight", weight, dn * xhat, edn * xhat.abs() + dn.abs() * ex),
                                 ("dbias", bias, dn, edn)):
        if p is None:
            continue
        over = (0, 1) if p.dim() == 1 else (0,)
        rows = T * (G if p.dim() == 1 else 1)
        res[name] = term.sum(over)
        res[name + "_bound"] = eterm.sum(over) + term.abs().sum(over) * (rows / 64 + 64) * U
    return res
