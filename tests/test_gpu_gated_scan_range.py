"""The gated linear recurrence over the whole range of its decays on long axes, in few channel blocks (the states
go through groups of tiles) and in more: growing states, decays that are not finite, dropped states (needs a gfx950
GPU).  Tolerances are the oracle's element-wise bounds plus the stored type's rounding."""
import math

import pytest
import torch

from oracle import layers
from tests.test_gpu_gated_scan import F32, close, gdp  # noqa: F401

pytestmark = pytest.mark.gpu


def oracle(x, g, cut, s0, d_o, d_final, complement):
    """The oracle's values, with its bounds widened by the steps of subnormal results, which its relative ones do
    not hold: a row's result, and those of its wave, its tile and its group, are each rounded by at most 2^-150
    there, and what that changes follows the recurrence."""
    ref = layers.scan(x, g, cut, s0, complement)
    want = layers.scan_backward(x, g, cut, d_o, d_final, s0, complement)
    step = layers.scan(torch.full_like(x, 4 * 2.0 ** -150, dtype=torch.float64), g, cut)
    back = layers.scan_backward(x, g, cut, torch.full_like(x, 4 * 2.0 ** -150, dtype=torch.float64), None, None)
    e = layers.scan_backward(x, g, cut, d_o.abs(), None if d_final is None else d_final.abs(), None)["dx"]
    p = layers.scan(x.abs(), g, cut, None if s0 is None else s0.abs())["before"] + (x.abs() if complement else 0)
    a = g.double().exp()
    ref["o_bound"] += step["o"]
    ref["final_bound"] += step["final"]
    want["dx_bound"] += back["dx"] * (torch.expm1(g.double()).abs() if complement else 1)
    want["dg_bound"] += a * (e * step["before"] + back["dx"] * p) + e * 2.0 ** -150
    want["ds0_bound"] += a[[min(c, len(a) - 1) for c in cut[:-1]]] * back["dx"][[min(c, len(a) - 1) for c in cut[:-1]]]
    return ref, want


def compare(gdp, x, g, cu, s0, d_o, d_final, complement=False):  # noqa: F811
    """Forward pass and gradients (with the forward's checkpoints, and without) against the oracle."""
    cut, xd, gd, cud = cu.tolist(), x.cuda(), g.cuda(), cu.cuda()
    sd, dd, fd = (None if t is None else t.cuda() for t in (s0, d_o, d_final))
    ref, want = oracle(x, g, cut, s0, d_o, d_final, complement)
    assert all(torch.isfinite(t.float()).all() for t in (*ref.values(), *want.values())), "the case leaves float32"
    o, fs, points = gdp.gated_scan(xd, gd, cud, initial_state=sd, output_final_state=True, complement_input=complement,
                                   return_checkpoints=True)
    close(o, ref["o"], ref["o_bound"], ("o", x.dtype))
    close(fs, ref["final"], ref["final_bound"], ("final", F32))
    for cp in (points, None):
        r = gdp.gated_scan_backward(xd, gd, cud, dd, d_final_state=fd, initial_state=sd, complement_input=complement,
                                    checkpoints=cp)
        close(r["dx"], want["dx"], want["dx_bound"], ("dx", F32))
        close(r["dg_log"], want["dg"], want["dg_bound"], ("dg", F32))
        if s0 is not None:
            close(r["d_initial_state"], want["ds0"], want["ds0_bound"], ("ds0", F32))


# D: one channel block, four of them (both through groups of tiles), five
CHANNELS = [6, 512, 600]


@pytest.mark.parametrize("D", CHANNELS)
@pytest.mark.parametrize("initial", [False, True])
@pytest.mark.parametrize("complement", [False, True])
def test_growth_of_nothing_is_nothing(gdp, D, initial, complement):  # noqa: F811
    """Positive log decays, 128 rows of which multiply to a float32, over states (and gradients) of zero: the
    products over thousands of rows pass float32, the results are zeros."""
    lens = [8192, 700]
    rates = torch.linspace(0.047, 0.69, D)
    g = rates.expand(sum(lens), D).contiguous()
    x = torch.zeros_like(g)
    s0 = torch.zeros(2, D) if initial else None
    cu = torch.tensor([0, 8192, 8892], dtype=torch.int32, device="cuda")
    o, fs, points = gdp.gated_scan(x.cuda(), g.cuda(), cu, initial_state=None if s0 is None else s0.cuda(),
                                   output_final_state=True, return_checkpoints=True, complement_input=complement)
    assert not o.any() and not fs.any()
    for cp in (points, None):
        r = gdp.gated_scan_backward(x.cuda(), g.cuda(), cu, x.cuda(), checkpoints=cp, complement_input=complement,
                                    initial_state=None if s0 is None else s0.cuda())
        for name, v in r.items():
            assert v is None or not v.any(), name


def swing(T, rates, nats):
    """Log decays +rate, then -rate, for `nats` / rate rows each, per channel."""
    half = (nats / rates).floor().long()
    up = (torch.arange(T)[:, None] // half) % 2 == 0
    return torch.where(up, rates, -rates)


@pytest.mark.parametrize("D", CHANNELS)
@pytest.mark.parametrize("lens,first,behind", [([9300, 100, 2700], 0, 0), ([2048, 4200, 5000], 70, 90)])
@pytest.mark.parametrize("complement", [False, True])
def test_small_states_that_grow_and_shrink(gdp, D, lens, first, behind, complement):  # noqa: F811
    """States of 1e-30 that grow to 1e26 and come back, again and again: the products of decays over the rows of a
    group pass float32 in both directions, those over 128 rows do not, nor do the states."""
    gen = torch.Generator().manual_seed(D)
    T, N = first + sum(lens) + behind, len(lens)
    cu = torch.tensor([first] + [first + sum(lens[:i + 1]) for i in range(N)], dtype=torch.int32)
    g = swing(T, torch.linspace(0.047, 0.6, D), 130.0)
    x, d_o = (1e-31 * torch.randn(T, D, generator=gen) for _ in range(2))
    s0, d_final = (1e-30 * torch.randn(N, D, generator=gen) for _ in range(2))
    compare_outside(gdp, x, g, cu, s0, d_o, d_final, complement)


def compare_outside(gdp, x, g, cu, s0, d_o, d_final, complement):  # noqa: F811
    """compare, with the rows that no sequence covers left out of the forward pass's outputs."""
    lo, hi = int(cu[0]), int(cu[-1])
    part = slice(lo, hi)
    if lo == 0 and hi == x.shape[0]:
        return compare(gdp, x, g, cu, s0, d_o, d_final, complement)
    ref, want = oracle(x, g, cu.tolist(), s0, d_o, d_final, complement)
    o, fs = gdp.gated_scan(x.cuda(), g.cuda(), cu.cuda(), initial_state=s0.cuda(), output_final_state=True,
                           complement_input=complement)
    close(o[part], ref["o"][part], ref["o_bound"][part], ("o", x.dtype))
    close(fs, ref["final"], ref["final_bound"], ("final", F32))
    r = gdp.gated_scan_backward(x.cuda(), g.cuda(), cu.cuda(), d_o.cuda(), d_final_state=d_final.cuda(),
                                initial_state=s0.cuda(), complement_input=complement)
    close(r["dx"], want["dx"], want["dx_bound"], ("dx", F32))
    close(r["dg_log"], want["dg"], want["dg_bound"], ("dg", F32))
    close(r["d_initial_state"], want["ds0"], want["ds0_bound"], ("ds0", F32))


@pytest.mark.parametrize("D", [6, 600])
def test_a_large_state_comes_back_from_far_below(gdp, D):  # noqa: F811
    """A state of 1e25 without any input that shrinks by e^-110 over 2048 rows and grows again: what is left of it
    there is a float32, though the product of its decays is not."""
    T = 4 * 2048 + 300
    rate = 110.0 / 2048
    g = swing(T, torch.full((D,), -rate), -110.0)
    x = torch.zeros(T, D)
    s0 = 1e25 * (1 + torch.rand(1, D, generator=torch.Generator().manual_seed(3)))
    cu = torch.tensor([0, T], dtype=torch.int32)
    assert math.isclose(float(g[:2048].double().sum(0)[0]), -110, rel_tol=1e-2)
    compare(gdp, x, g, cu, s0, x, 1e-16 * torch.ones(1, D))


@pytest.mark.parametrize("D", [40, 600])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 100.0])
def test_a_bad_gate_stays_in_its_sequence_over_groups(gdp, D, bad):  # noqa: F811
    """A decay that is not finite, a group of tiles and more before its sequence's end (which lies at a group's end
    and inside one): no other sequence or channel sees it, to the bit."""
    gen = torch.Generator().manual_seed(31)
    lens = [6144, 5000, 4700]
    T, N = sum(lens), 3
    cu = torch.tensor([0, 6144, 11144, 15844], dtype=torch.int32).cuda()
    x, d_o = (torch.randn(T, D, generator=gen).cuda() for _ in range(2))
    g = (-torch.nn.functional.softplus(torch.randn(T, D, generator=gen) - 3)).cuda()
    s0, d_final = (torch.randn(N, D, generator=gen).cuda() for _ in range(2))
    worse = g.clone()
    worse[1000, 3] = bad
    worse[7000, 5] = bad
    got = []
    for gates in (g, worse):
        o, fs, points = gdp.gated_scan(x, gates, cu, initial_state=s0, output_final_state=True, return_checkpoints=True)
        r = gdp.gated_scan_backward(x, gates, cu, d_o, d_final_state=d_final, initial_state=s0, checkpoints=points)
        got.append({"o": o, "fs": fs, **r})
    good, poor = got
    rows = torch.ones(T, D, dtype=torch.bool)
    rows[:6144, 3] = False
    rows[6144:11144, 5] = False
    states = torch.ones(N, D, dtype=torch.bool)
    states[0, 3] = states[1, 5] = False
    for name, value in good.items():
        where = (states if name in ("fs", "d_initial_state") else rows).cuda()
        assert torch.equal(poor[name][where], value[where]), name


@pytest.mark.parametrize("D", [64, 576])
@pytest.mark.parametrize("complement", [False, True])
def test_extreme_gates_over_groups(gdp, D, complement):  # noqa: F811
    """-inf restarts a channel, 0 keeps a running sum, strong decays underflow, a channel without input, on an axis
    of several groups."""
    gen = torch.Generator().manual_seed(11)
    lens = [5000, 3200]
    T = sum(lens)
    x = torch.randn(T, D, generator=gen)
    g = -torch.nn.functional.softplus(torch.randn(T, D, generator=gen) - 3)
    q = D // 4
    g[:, :q] = 0.0
    g[:, 2 * q:3 * q] *= 400.0
    g.clamp_(min=-700.0)  # further down the bound of exp is no float64
    g[::1500, q:2 * q] = float("-inf")
    x[:, 3 * q:3 * q + 3] = 0.0
    cu = torch.tensor([0, 5000, 8200], dtype=torch.int32)
    s0 = torch.randn(2, D, generator=gen)
    compare(gdp, x, g, cu, s0, torch.randn(T, D, generator=gen), torch.randn(2, D, generator=gen), complement)
