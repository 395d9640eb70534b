"""float64 oracle of the short convolution, of the selective scan and of the norms around a block, with error bounds.

Test infrastructure only: the definitions in torch float64 on the CPU, sharing no
code with the GPU path.  Next to each value stands a bound on the error of a
float32 evaluation of the same formula, to first order in U = 2^-24 (half a step
of float32, relative), counted rounding by rounding: a product or a sum adds U of
its value, a sum of n products n + 1 U of the sum of their magnitudes, and an
operand's own bound is carried on with what multiplies it.  The exponential, the
sigmoid and the activations count as in oracle/layers.py.

  softplus(v) = max(v, 0) + log(1 + e), e = exp(-|v|): e is off by (2 |v| + 4) U
      relative, which log(1 + e) carries on with a factor of at most 1; e / (2 + e)
      adds 4 U (a sum, a reciprocal good to one step, a product), the polynomial in
      its square 3 U and what its rounded coefficients leave 1/2 U, the last product U:
      (2 |v| + 14) U of log(1 + e) at most, and U of the sum;
  exp(delta A): the product delta A log2(e) is rounded twice and its constant once
      (3 U of |delta A|), the exponential good to one step (2 U, one to spare); a
      value below 2^-126 may come out as 0;
  the joined decay over a chunk, exp(A sum delta): the sum of n steps in parts of
      four is off by at most (n / 4 + 4) U of itself; `join` is that number, 64 for
      chunks of up to 240 rows.  Its share of a state is counted row by row.
Sums over tokens run in chunks of up to `chain` rows one after another, then over
the chunks 64 apart and pairwise: a sum of n rows in that order is off by at most
chain + (number of chunks) / 64 + 1 + 6 additions' U of the magnitudes' sum.  The rows per
chunk follow from the sizes as the library's do (conv_chunk_rows, select_chunk_rows; the
sizes of its workspaces tell them).  Everything is doubled for the second order.
"""
import torch

from .layers import U, F64, _activation, rounded  # noqa: F401  (rounded: for the tests)

TINY = 2.0 ** -126


def _cpu(t):
    return None if t is None else t.detach().cpu().to(F64)


def _edges(cu):
    return [int(c) for c in cu]


def _chunk_rows(T, blocks, want, least, most):
    """The longest chunks of 2^least to 2^most rows of which there are `want` in all channel blocks."""
    shift = most
    while shift > least and (T >> shift) * blocks < want:
        shift -= 1
    return 1 << shift


def conv_chunk_rows(T, D):
    """Rows per chunk of the convolution's gradients."""
    return _chunk_rows(T, -(-D // 64), 4096, 4, 7)


def select_chunk_rows(T, N, D, G):
    """Rows per chunk of the scan, forward and in the gradients."""
    blocks = G * -(-(D // G) // 64)
    rows = _chunk_rows(T, blocks, 4096, 4, 11)
    if N * blocks >= 2048:
        while rows < 2048 and rows * N < 2 * T:
            rows *= 2
    return rows, _chunk_rows(T, blocks, 2048, 6, 11)


# the residual norm's gradients: workgroups at most, each with its own partial sums
NORM_WORKGROUPS = 512


# ------------------------------------------------------------ short convolution

def conv(x, weight, cu, bias=None, activation=None, s0=None, d_y=None, d_final=None):
    """y, final [N, W-1, D] (exact) and, with d_y, dx, dweight, dbias, ds0; bounds beside them."""
    x, w, b, s0, d_y, d_final = (_cpu(t) for t in (x, weight, bias, s0, d_y, d_final))
    T, D = x.shape
    W = w.shape[1]
    edges = _edges(cu)
    N = len(edges) - 1
    slope_max = {"silu": 1.1, "sigmoid": 0.25}.get(activation, 1.0)   # of act
    curve_max = {"silu": 0.5, "sigmoid": 0.1}.get(activation, 0.0)    # of act'
    res = {"final": torch.zeros(N, W - 1, D, dtype=F64)}
    for name, like in (("y", x), ("dx", x), ("dweight", w), ("dbias", w[:, 0]), ("ds0", res["final"])):
        res[name], res[name + "_bound"] = torch.zeros_like(like), torch.zeros_like(like)
    mag_w, mag_b = torch.zeros_like(w), torch.zeros_like(w[:, 0])
    for i, (lo, hi) in enumerate(zip(edges, edges[1:])):
        n = max(hi - lo, 0)
        rows = torch.cat([torch.zeros(W - 1, D, dtype=F64) if s0 is None else s0[i], x[lo:lo + n]])
        res["final"][i] = rows[n:]
        v = torch.zeros(n, D, dtype=F64) if b is None else b.expand(n, D).clone()
        mag = v.abs()
        for j in range(W):
            v = v + w[:, j] * rows[j:j + n]
            mag = mag + (w[:, j] * rows[j:j + n]).abs()
        ev = (W + 1) * U * mag
        f, df, ef, edf = _activation(activation, v)
        res["y"][lo:lo + n], res["y_bound"][lo:lo + n] = f, 2 * (ef + slope_max * ev)
        if d_y is None:
            continue
        g = d_y[lo:lo + n]
        dv = g * df
        edv = g.abs() * (edf + curve_max * ev) + dv.abs() * U
        drows, erows, mrows = (torch.zeros_like(rows) for _ in range(3))
        for j in range(W):
            drows[j:j + n] += w[:, j] * dv
            erows[j:j + n] += w[:, j].abs() * edv
            mrows[j:j + n] += (w[:, j] * dv).abs()
            res["dweight"][:, j] += (dv * rows[j:j + n]).sum(0)
            res["dweight_bound"][:, j] += (edv * rows[j:j + n].abs()).sum(0)
            mag_w[:, j] += (dv * rows[j:j + n]).abs().sum(0)
        res["dbias"] += dv.sum(0)
        res["dbias_bound"] += edv.sum(0)
        mag_b += dv.abs().sum(0)
        if d_final is not None:
            drows[n:] += d_final[i]
            mrows[n:] += d_final[i].abs()
        erows = 2 * (erows + (W + 2) * U * mrows)
        res["ds0"][i], res["ds0_bound"][i] = drows[:W - 1], erows[:W - 1]
        res["dx"][lo:lo + n], res["dx_bound"][lo:lo + n] = drows[W - 1:], erows[W - 1:]
    chunk = conv_chunk_rows(T, D)
    chain = (chunk + (T / chunk + N) / 64 + 8) * U
    res["dweight_bound"] = 2 * (res["dweight_bound"] + chain * mag_w)
    res["dbias_bound"] = 2 * (res["dbias_bound"] + chain * mag_b)
    return res


def conv_decode(x, weight, cache, slots, bias=None, activation=None):
    x, w, new = _cpu(x), _cpu(weight), _cpu(cache).clone()
    y, yb = torch.zeros_like(x), torch.zeros_like(x)
    for i, s in enumerate(int(s) for s in slots):
        if 0 <= s < new.shape[0]:
            r = conv(x[i:i + 1], w, [0, 1], bias, activation, new[s:s + 1])
            y[i], yb[i], new[s] = r["y"][0], r["y_bound"][0], r["final"][0]
    return {"y": y, "y_bound": yb, "cache": new}


# --------------------------------------------------------------- selective scan

def _steps(dt, bias, softplus):
    """delta, d delta / d dt and their bounds."""
    v = dt if bias is None else dt + bias
    ev = v.abs() * U if bias is not None else torch.zeros_like(v)
    if not softplus:
        return v, torch.ones_like(v), ev, torch.zeros_like(v)
    tail = torch.log1p(torch.exp(-v.abs()))
    delta = v.clamp(min=0) + tail
    slope, _, es, _ = _activation("sigmoid", v)
    return delta, slope, slope * ev + tail * (2 * v.abs() + 14) * U + delta * U + TINY, es + 0.25 * ev


def select(u, dt, A, B, C, cu, skip=None, gate=None, dt_bias=None, dt_softplus=False, s0=None, d_o=None, d_final=None,
           join=64, chain=64):
    """o, final [N, D, S] and, with d_o, all gradients; bounds beside them.  Sequences run side by side."""
    u, dt, A, B, C, skip, z, bias, s0, d_o, d_final = (
        _cpu(t) for t in (u, dt, A, B, C, skip, gate, dt_bias, s0, d_o, d_final))
    (T, D), S, G = u.shape, A.shape[1], B.shape[1]
    edges = _edges(cu)
    N = len(edges) - 1
    rows, rows_back = select_chunk_rows(T, N, D, G)
    assert max(rows, rows_back) / 4 + 4 <= join and rows_back <= chain, "the bounds are of shorter chunks"
    per = D // G
    wide = lambda t: t.repeat_interleave(per, 1)  # noqa: E731  [rows, G, S] -> [rows, D, S]
    narrow = lambda t: t.unflatten(1, (G, per)).sum(2)  # noqa: E731
    skip = torch.zeros(D, dtype=F64) if skip is None else skip
    delta, slope, ed, es = _steps(dt, bias, dt_softplus)
    w = delta * u
    ew = u.abs() * ed + w.abs() * U
    f, df, ef, edf = _activation("silu", z) if z is not None else (torch.ones_like(u), *[torch.zeros_like(u)] * 3)
    order = sorted(range(N), key=lambda i: edges[i] - edges[i + 1])
    sizes = [max(edges[i + 1] - edges[i], 0) for i in order]
    rank, start = torch.tensor(order, dtype=torch.long), torch.tensor([edges[i] for i in order], dtype=torch.long)
    live = lambda t: sum(n > t for n in sizes)  # noqa: E731

    def decays(rows):
        a = (delta[rows, :, None] * A).exp()
        x = (delta[rows, :, None] * A).abs()
        ea = A.abs() * ed[rows, :, None] + x * 3 * U + 3 * U
        return a, torch.where(a > 0, ea + TINY / a, torch.zeros_like(a)), x

    zero = torch.zeros(N, D, S, dtype=F64)
    h, b = (zero.clone() if s0 is None else s0[rank].clone()), zero.clone()
    pre, epre = torch.zeros_like(u), torch.zeros_like(u)
    back = d_o is not None
    before, bbefore = (torch.zeros(T, D, S, dtype=F64) for _ in range(2)) if back else (None, None)
    for t in range(max(sizes, default=0)):
        k = live(t)
        rows = start[:k] + t
        if back:
            before[rows], bbefore[rows] = h[:k], b[:k]
        a, ea, x = decays(rows)
        Bw, Cw = wide(B[rows]), wide(C[rows])
        carried, term = a * h[:k], w[rows, :, None] * Bw
        b[:k] = a * b[:k] + carried.abs() * (ea + x * join * U) + ew[rows, :, None] * Bw.abs() + term.abs() * U
        h[:k] = carried + term
        b[:k] += h[:k].abs() * U
        pre[rows] = (Cw * h[:k]).sum(-1) + skip * u[rows]
        epre[rows] = (Cw.abs() * b[:k]).sum(-1) + ((Cw * h[:k]).abs().sum(-1) + (skip * u[rows]).abs()) * (S + 2) * U
    final, fb = torch.zeros_like(h), torch.zeros_like(b)
    final[rank], fb[rank] = h, b
    o = pre * f
    res = {"o": o, "o_bound": 2 * (epre * f.abs() + pre.abs() * ef + o.abs() * U), "final": final, "final_bound": 2 * fb}
    if not back:
        return res
    gy = d_o * f
    egy = d_o.abs() * ef + gy.abs() * U
    e, b = (zero.clone() if d_final is None else d_final[rank].clone()), zero.clone()
    end = start + torch.tensor(sizes, dtype=torch.long) - 1
    names = ("through", "ethrough", "carried", "ecarried")
    acc = {n: torch.zeros_like(u) for n in names}
    dB, eB, dC, eC = (torch.zeros_like(B) for _ in range(4))
    dA, eA, magA = (torch.zeros_like(A) for _ in range(3))
    lanes = (8 + per / 64) * U
    for t in range(max(sizes, default=0)):
        k = live(t)
        rows = end[:k] - t
        a, ea, x = decays(rows)
        Bw, Cw, g, eg = wide(B[rows]), wide(C[rows]), gy[rows, :, None], egy[rows, :, None]
        e[:k] += Cw * g
        b[:k] += Cw.abs() * eg + (Cw * g).abs() * U + e[:k].abs() * U
        hb, bb = before[rows], bbefore[rows]
        term = w[rows, :, None] * Bw
        after = a * hb + term
        bafter = a * bb + (a * hb).abs() * (ea + U) + ew[rows, :, None] * Bw.abs() + (term.abs() + after.abs()) * U
        dC[rows] = narrow(g * after)
        eC[rows] = narrow(g.abs() * bafter + eg * after.abs()) + narrow((g * after).abs()) * (lanes + U)
        wr, er = w[rows, :, None], ew[rows, :, None]
        dB[rows] = narrow(e[:k] * wr)
        eB[rows] = narrow(b[:k] * wr.abs() + e[:k].abs() * er) + narrow((e[:k] * wr).abs()) * (lanes + U)
        acc["through"][rows] = (e[:k] * Bw).sum(-1)
        acc["ethrough"][rows] = (b[:k] * Bw.abs()).sum(-1) + (e[:k] * Bw).abs().sum(-1) * (S + 2) * U
        c = e[:k] * a * hb
        ec = a * (b[:k] * hb.abs() + e[:k].abs() * bb) + c.abs() * (ea + 3 * U)
        acc["carried"][rows] = (c * A).sum(-1)
        acc["ecarried"][rows] = (ec * A.abs()).sum(-1) + (c * A).abs().sum(-1) * (S + 2) * U
        dl, edl = delta[rows, :, None], ed[rows, :, None]
        dA += (c * dl).sum(0)
        eA += (ec * dl.abs() + c.abs() * edl).sum(0)
        magA += (c * dl).abs().sum(0)
        b[:k] = a * b[:k] + (a * e[:k]).abs() * (ea + U + x * join * U)
        e[:k] *= a
    ds0, eds0 = torch.zeros_like(e), torch.zeros_like(b)
    ds0[rank], eds0[rank] = e, b
    inside = torch.zeros(T, 1, dtype=F64)
    for lo, hi in zip(edges, edges[1:]):
        inside[lo:hi] = 1
    thr, ethr, car, ecar = (acc[n] for n in names)
    du = (skip * gy + delta * thr) * inside
    edu = skip.abs() * egy + ed * thr.abs() + delta.abs() * ethr + 3 * U * ((skip * gy).abs() + (delta * thr).abs())
    dd = u * thr + car
    edd = u.abs() * ethr + ecar + 2 * U * ((u * thr).abs() + car.abs())
    ddt = dd * slope * inside
    eddt = dd.abs() * es + slope.abs() * edd + ddt.abs() * U
    dz = d_o * df * pre * inside
    edz = d_o.abs() * (edf * pre.abs() + df.abs() * epre) + dz.abs() * 3 * U
    sums = (chain + (T / 64 + N) / 64 + 16) * U
    res.update(
        du=du, du_bound=2 * edu, ddt=ddt, ddt_bound=2 * eddt, dB=dB, dB_bound=2 * eB, dC=dC, dC_bound=2 * eC, dA=dA,
        dA_bound=2 * (eA + magA * (sums + 2 * U)), dskip=(gy * u * inside).sum(0),
        dskip_bound=2 * ((egy * u.abs()).sum(0) + (gy * u).abs().sum(0) * (sums + U)), dgate=dz, dgate_bound=2 * edz,
        ddt_bias=ddt.sum(0), ddt_bias_bound=2 * ((eddt * inside).sum(0) + ddt.abs().sum(0) * sums), ds0=ds0,
        ds0_bound=2 * eds0)
    return res


def select_decode(u, dt, A, B, C, cache, slots, **form):
    new = _cpu(cache).clone()
    o, ob, cb = torch.zeros(u.shape, dtype=F64), torch.zeros(u.shape, dtype=F64), torch.zeros_like(new)
    gate = form.pop("gate", None)
    for i, s in enumerate(int(s) for s in slots):
        if 0 <= s < new.shape[0]:
            one = slice(i, i + 1)
            r = select(u[one], dt[one], A, B[one], C[one], [0, 1], gate=None if gate is None else gate[one],
                       s0=new[s:s + 1], **form)
            o[i], ob[i], new[s], cb[s] = r["o"][0], r["o_bound"][0], r["final"][0], r["final_bound"][0]
    return {"o": o, "o_bound": ob, "cache": new, "cache_bound": cb}


# ---------------------------------------------------------- norms around a block

def residual_norm(x, y, post_weight=None, pre_weight=None, gate=None, activation=None, post_norm=True, pre_norm=True,
                  residual_scale=1.0, eps=1e-5, d_r=None, d_n=None):
    """r, n (and with d_r or d_n the gradients dx, dy, dgate, dpost_weight, dpre_weight), with bounds.  A sum over the
    channels runs over at most 16 of them, 6 steps between lanes and 16 waves: S = 40 U of the magnitudes' sum."""
    x, y, wa, wb, z, d_r, d_n = (_cpu(t) for t in (x, y, post_weight, pre_weight, gate, d_r, d_n))
    T, D = y.shape
    S, c = 40 * U, float(torch.tensor(residual_scale, dtype=torch.float32))
    eps = float(torch.tensor(eps, dtype=torch.float32))
    wa = torch.ones(D, dtype=F64) if wa is None else wa
    wb = torch.ones(D, dtype=F64) if wb is None else wb
    mean = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    f, df, ef, edf = _activation(activation, z) if z is not None else (torch.ones_like(y), *[torch.zeros_like(y)] * 3)
    if post_norm:
        var = mean(y * y)
        ry = (var + eps) ** -0.5
        ery = 0.5 * var * (S + 2 * U) / (var + eps) + 4 * U  # relative
        yhat, eyh = y * ry, (y * ry).abs() * (ery + U)
    else:
        ry, ery, yhat, eyh = torch.ones(T, 1, dtype=F64), torch.zeros(T, 1, dtype=F64), y, torch.zeros_like(y)
    p = c * yhat * wa * f
    ep = abs(c) * wa.abs() * (eyh * f.abs() + yhat.abs() * ef) + p.abs() * 3 * U
    r = x + p
    er = ep + r.abs() * U
    res = {"r": r, "r_bound": 2 * er}
    if pre_norm:
        var = mean(r * r)
        rr = (var + eps) ** -0.5
        err = 0.5 * (2 * mean(r.abs() * er) + var * (S + 2 * U)) / (var + eps) + 4 * U
        rhat = r * rr
        erh = er * rr + rhat.abs() * (err + U)
        res["n"], res["n_bound"] = rhat * wb, 2 * (erh * wb.abs() + 2 * U * (rhat * wb).abs())
    if d_r is None and d_n is None:
        return res
    # a team's rows one after another, then up to 256 teams of a workgroup, then the workgroups' sums (of wide
    # rows two teams' each) 64 apart and pairwise
    rows = (T / NORM_WORKGROUPS + 1 + 256 + 2 * NORM_WORKGROUPS / 64 + 8) * U
    e = torch.zeros_like(x) if d_r is None else d_r
    ee = torch.zeros_like(x)
    if pre_norm:
        q = d_n * wb
        s = mean(q * rhat)
        ems = mean(q.abs() * erh) + mean((q * rhat).abs()) * (S + 3 * U)
        inner = q - rhat * s
        einner = q.abs() * U + erh * s.abs() + rhat.abs() * ems + 2 * U * (q.abs() + (rhat * s).abs())
        e = e + rr * inner
        ee = rr * einner + (rr * inner).abs() * (err + U) + e.abs() * U
        res["dpre_weight"] = (d_n * rhat).sum(0)
        res["dpre_weight_bound"] = 2 * ((d_n.abs() * erh).sum(0) + (d_n * rhat).abs().sum(0) * (rows + U))
    res["dx"], res["dx_bound"] = e, 2 * ee
    d, ed = c * e, abs(c) * ee + (c * e).abs() * U
    if z is not None:
        g = yhat * wa * df
        eg = wa.abs() * (eyh * df.abs() + yhat.abs() * edf) + 2 * U * g.abs()
        res["dgate"], res["dgate_bound"] = d * g, 2 * (d.abs() * eg + ed * g.abs() + (d * g).abs() * 2 * U)
    dp, edp = d * f, d.abs() * ef + ed * f.abs() + (d * f).abs() * U
    res["dpost_weight"] = (dp * yhat).sum(0)
    res["dpost_weight_bound"] = 2 * ((edp * yhat.abs() + dp.abs() * eyh).sum(0) + (dp * yhat).abs().sum(0) * (rows + U))
    v, ev = dp * wa, edp * wa.abs() + (dp * wa).abs() * U
    if post_norm:
        s = mean(v * yhat)
        ems = mean(ev * yhat.abs() + v.abs() * eyh) + mean((v * yhat).abs()) * (S + 2 * U)
        inner = v - yhat * s
        einner = ev + eyh * s.abs() + yhat.abs() * ems + 2 * U * (v.abs() + (yhat * s).abs())
        dy, edy = ry * inner, ry * einner + (ry * inner).abs() * (ery + 2 * U)
    else:
        dy, edy = v, ev
    res["dy"], res["dy_bound"] = dy, 2 * edy
    return res
