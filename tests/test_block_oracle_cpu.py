"""The float64 oracle of the short convolution, the selective scan and the norms around a block against autograd on
the definitions and against differences (no GPU)."""
import pytest
import torch

from oracle import blocks

F64 = torch.float64


def randn(gen, *shape):
    return torch.randn(*shape, generator=gen, dtype=F64)


def act(name, v):
    return {None: lambda: v, "silu": lambda: v * torch.sigmoid(v), "sigmoid": lambda: torch.sigmoid(v)}[name]()



def differences(loss, t, grad, gen, step=1e-6):
    """The derivative of loss() along a random direction of t against the gradient."""
    d = randn(gen, *t.shape)
    with torch.no_grad():
        t += step * d
        hi = loss()
        t -= 2 * step * d
        lo = loss()
        t += step * d
    want = (grad * d).sum()
    assert abs((hi - lo) / (2 * step) - want) <= 1e-6 * (1 + want.abs() + hi.abs()), (hi, lo, want)


@pytest.mark.parametrize("activation", [None, "silu", "sigmoid"])
@pytest.mark.parametrize("W", [2, 4, 8])
def test_conv(activation, W):
    gen = torch.Generator().manual_seed(W)
    cu, D = [0, 1, 4, 4, 17], 5
    x, w, b = randn(gen, 17, D).requires_grad_(), randn(gen, D, W).requires_grad_(), randn(gen, D).requires_grad_()
    s0 = randn(gen, 4, W - 1, D).requires_grad_()
    dy, df = randn(gen, 17, D), randn(gen, 4, W - 1, D)

    def run():
        ys, fs = [], []
        for i in range(4):
            rows = torch.cat([s0[i], x[cu[i]:cu[i + 1]]])
            for t in range(cu[i + 1] - cu[i]):
                ys.append(act(activation, (rows[t:t + W].t() * w).sum(1) + b))
            fs.append(rows[len(rows) - (W - 1):])
        return torch.stack(ys), torch.stack(fs)

    y, fs = run()
    r = blocks.conv(x, w, cu, b, activation, s0, dy, df)
    assert torch.allclose(r["y"], y) and torch.equal(r["final"], fs)
    g = torch.autograd.grad((y * dy).sum() + (fs * df).sum(), (x, w, b, s0))
    for name, want in zip(("dx", "dweight", "dbias", "ds0"), g):
        assert torch.allclose(r[name], want, atol=1e-12), name
    loss = lambda: sum((o * d).sum() for o, d in zip(run(), (dy, df)))  # noqa: E731
    for t, name in ((x, "dx"), (w, "dweight"), (b, "dbias"), (s0, "ds0")):
        differences(loss, t, r[name], gen)
    c = blocks.conv_decode(x[:3], w, s0[:2], [1, -1, 0], b, activation)
    one = blocks.conv(x[2:3], w, [0, 1], b, activation, s0[:1])
    assert torch.equal(c["y"][2], one["y"][0]) and torch.equal(c["cache"][0], one["final"][0]) and (c["y"][1] == 0).all()


@pytest.mark.parametrize("gated,softplus,groups", [(True, True, 1), (False, False, 2), (True, False, 3)])
def test_select(gated, softplus, groups):
    gen = torch.Generator().manual_seed(groups)
    cu, T, D, S = [0, 1, 6, 6, 15], 15, 6, 3
    u, B, C = randn(gen, T, D), randn(gen, T, groups, S), randn(gen, T, groups, S)
    dt = randn(gen, T, D) if softplus else randn(gen, T, D).abs()
    A, skip, z = -randn(gen, D, S).abs(), randn(gen, D), randn(gen, T, D) if gated else None
    bias, s0 = randn(gen, D).abs(), randn(gen, 4, D, S)
    do, df = randn(gen, T, D), randn(gen, 4, D, S)
    leaves = [t.requires_grad_() for t in (u, dt, A, B, C, skip, bias, s0) + ((z,) if gated else ())]

    def run():
        delta = torch.nn.functional.softplus(dt + bias) if softplus else dt + bias
        os, fs = [], []
        for i in range(4):
            h = s0[i]
            for t in range(cu[i], cu[i + 1]):
                Bt, Ct = (p[t].repeat_interleave(D // groups, 0) for p in (B, C))
                h = torch.exp(delta[t][:, None] * A) * h + (delta[t] * u[t])[:, None] * Bt
                o = (h * Ct).sum(1) + skip * u[t]
                os.append(o * act("silu", z[t]) if gated else o)
            fs.append(h)
        return torch.stack(os), torch.stack(fs)

    o, fs = run()
    r = blocks.select(u, dt, A, B, C, cu, skip, z, bias, softplus, s0, do, df)
    assert torch.allclose(r["o"], o) and torch.allclose(r["final"], fs)
    names = ("du", "ddt", "dA", "dB", "dC", "dskip", "ddt_bias", "ds0") + (("dgate",) if gated else ())
    for name, want in zip(names, torch.autograd.grad((o * do).sum() + (fs * df).sum(), leaves)):
        assert torch.allclose(r[name], want, atol=1e-12), name
    loss = lambda: sum((a * d).sum() for a, d in zip(run(), (do, df)))  # noqa: E731
    for t, name in zip(leaves, names):
        differences(loss, t, r[name], gen)
    step = blocks.select_decode(u[:2], dt[:2], A, B[:2], C[:2], s0[:2], [1, 7], skip=skip, dt_bias=bias,
                                dt_softplus=softplus, gate=z)
    one = blocks.select(u[:1], dt[:1], A, B[:1], C[:1], [0, 1], skip, None if z is None else z[:1], bias, softplus,
                        s0[1:2])
    assert torch.equal(step["o"][0], one["o"][0]) and torch.equal(step["cache"][1], one["final"][0])
    assert (step["o"][1] == 0).all() and torch.equal(step["cache"][0], s0[0])


@pytest.mark.parametrize("activation", [None, "silu", "sigmoid"])
@pytest.mark.parametrize("post,pre,gated", [(True, True, True), (True, False, True), (False, True, False), (False, True, True)])
def test_residual_norm(activation, post, pre, gated):
    gen = torch.Generator().manual_seed(3)
    T, D, c, eps = 4, 7, 0.5, 2.0 ** -17
    x, y, z, wa, wb = (randn(gen, T, D), randn(gen, T, D), randn(gen, T, D), randn(gen, D), randn(gen, D))
    dr, dn = randn(gen, T, D), randn(gen, T, D)
    if not pre:
        wb = dn = None
    leaves = [t.requires_grad_() for t in (x, y, z if gated else None, wa, wb) if t is not None]

    def run():
        p = y * ((y * y).mean(-1, keepdim=True) + eps) ** -0.5 if post else y
        p = p * wa
        r = x + c * (p * act(activation, z) if gated else p)
        return (r, r * ((r * r).mean(-1, keepdim=True) + eps) ** -0.5 * wb) if pre else (r,)

    out = run()
    res = blocks.residual_norm(x, y, wa, wb, z if gated else None, activation, post, pre, c, eps, dr, dn)
    for name, want in zip(("r", "n"), out):
        assert torch.allclose(res[name], want), name
    names = ["dx", "dy"] + (["dgate"] if gated else []) + ["dpost_weight"] + (["dpre_weight"] if pre else [])
    loss = lambda: sum((o * d).sum() for o, d in zip(run(), (dr, dn)))  # noqa: E731
    for t, name, want in zip(leaves, names, torch.autograd.grad(loss(), leaves)):
        assert torch.allclose(res[name], want, atol=1e-12), name
        differences(loss, t, res[name], gen)
