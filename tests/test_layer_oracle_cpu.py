"""The layers' float64 oracle against its own definitions differentiated: autograd and central
differences (no GPU)."""
import pytest
import torch

from oracle import layers

F64 = torch.float64


def _scan_loss(x, g, s0, cu, complement, d_o, d_final):
    loss = x.new_zeros(())
    for i in range(len(cu) - 1):
        h = s0[i]
        for t in range(cu[i], cu[i + 1]):
            a = torch.exp(g[t])
            h = a * h + ((1 - a) * x[t] if complement else x[t])
            loss = loss + (h * d_o[t]).sum()
        loss = loss + (h * d_final[i]).sum()
    return loss


@pytest.mark.parametrize("complement", [False, True])
def test_scan_gradients_against_autograd_and_differences(complement):
    gen = torch.Generator().manual_seed(1)
    cu = [0, 3, 3, 8, 9]
    T, N, D = 9, 4, 2
    x, d_o = torch.randn(T, D, generator=gen, dtype=F64), torch.randn(T, D, generator=gen, dtype=F64)
    g = -torch.rand(T, D, generator=gen, dtype=F64)
    s0, d_final = torch.randn(N, D, generator=gen, dtype=F64), torch.randn(N, D, generator=gen, dtype=F64)
    got = layers.scan_backward(x, g, cu, d_o, d_final, s0, complement)
    leaves = [t.clone().requires_grad_() for t in (x, g, s0)]
    _scan_loss(*leaves, cu, complement, d_o, d_final).backward()
    for leaf, name in zip(leaves, ("dx", "dg", "ds0")):
        assert torch.allclose(got[name], leaf.grad, rtol=1e-12, atol=1e-12), name
    step = 1e-5  # the third derivatives are of order 1: truncation below 1e-9
    for at, name in enumerate(("dx", "dg", "ds0")):
        args = [x, g, s0]
        for k in range(args[at].numel()):
            diff = []
            for sign in (1, -1):
                moved = [t.clone() for t in args]
                moved[at].view(-1)[k] += sign * step
                diff.append(_scan_loss(*moved, cu, complement, d_o, d_final))
            assert abs((diff[0] - diff[1]) / (2 * step) - got[name].view(-1)[k]) < 1e-8, (name, k)


@pytest.mark.parametrize("activation", [None, "silu", "sigmoid"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("shared", [False, True])
def test_norm_gradients_against_autograd_and_differences(activation, gated, center, shared):
    gen = torch.Generator().manual_seed(2)
    T, G, V = 3, 2, 5
    x, z, dy = (torch.randn(T, G, V, generator=gen, dtype=F64) for _ in range(3))
    shape = (V,) if shared else (G, V)
    w, b = (torch.randn(*shape, generator=gen, dtype=F64) for _ in range(2))

    def loss(x, w, b, z):
        d = x - x.mean(-1, keepdim=True) if center else x
        n = d / torch.sqrt((d * d).mean(-1, keepdim=True) + 1e-3) * w + b
        v = z if gated else n
        f = {None: lambda: v, "silu": lambda: v * torch.sigmoid(v), "sigmoid": lambda: torch.sigmoid(v)}[activation]()
        return ((n * f if gated else f) * dy).sum()

    got = layers.norm(x, w, b, z if gated else None, activation, center, 1e-3, dy)
    assert torch.allclose((got["y"] * dy).sum(), loss(x, w, b, z), rtol=1e-12)
    names = ("dx", "dweight", "dbias") + (("dgate",) if gated else ())
    leaves = [t.clone().requires_grad_() for t in (x, w, b, z)]
    loss(*leaves).backward()
    for leaf, name in zip(leaves, names):
        assert torch.allclose(got[name], leaf.grad, rtol=1e-11, atol=1e-12), name
    step = 1e-5
    for at, name in enumerate(names):
        for k in range(0, (x, w, b, z)[at].numel(), 3):
            diff = []
            for sign in (1, -1):
                moved = [t.clone() for t in (x, w, b, z)]
                moved[at].view(-1)[k] += sign * step
                diff.append(loss(*moved))
            assert abs((diff[0] - diff[1]) / (2 * step) - got[name].view(-1)[k]) < 1e-7, (name, k)


def test_a_plain_float32_evaluation_stays_within_the_bounds():
    """The bounds hold for the formulas evaluated in float32 in the simplest way."""
    gen = torch.Generator().manual_seed(3)
    x, g = torch.randn(200, 8, generator=gen), -torch.nn.functional.softplus(torch.randn(200, 8, generator=gen) - 2)
    f = layers.scan(x, g, [0, 70, 200])
    h = torch.zeros(8)
    for t in range(200):
        h = (torch.zeros(8) if t == 70 else h) * torch.exp(g[t]) + x[t]
        assert ((h.double() - f["o"][t]).abs() <= f["o_bound"][t]).all()
    y = torch.randn(6, 3, 40, generator=gen)
    r = layers.norm(y, activation="silu")
    n = (y - y.mean(-1, keepdim=True)) * torch.rsqrt(y.var(-1, unbiased=False, keepdim=True) + 1e-5)
    assert (((n * torch.sigmoid(n)).double() - r["y"]).abs() <= r["y_bound"]).all()
