"""The group norm and its gradients where groups are many and tokens few, and without a workspace (needs a gfx950
GPU)."""
import pytest
import torch

from oracle import layers
from tests.test_gpu_group_norm import BF16, F16, F32, check_norm, close, gdp, make  # noqa: F401

pytestmark = pytest.mark.gpu

SIZES = [(1, 4097, 128), (1, 65535, 8), (2, 65535, 1), (3, 1021, 100), (7, 769, 17), (2, 385, 520), (1, 771, 4104),
         (40, 1031, 8), (200, 511, 16), (13, 97, 2050)]


@pytest.mark.parametrize("T,G,V", SIZES)
@pytest.mark.parametrize("weight,bias", [("channel", True), ("head", False), ("none", True)])
def test_odd_numbers_of_groups(gdp, T, G, V, weight, bias):  # noqa: F811
    dtype = (F32, BF16, F16)[G % 3]
    check_norm(gdp, *make(T, G, V, dtype, weight=weight, bias=bias, gated=weight != "none", seed=G), "silu", V > 1)


@pytest.mark.parametrize("T,G,V", [(1, 4097, 128), (300, 7, 65)])
def test_no_parameters_and_no_workspace(gdp, T, G, V):  # noqa: F811
    x, _, _, z, dy = make(T, G, V, F32, weight="none", seed=8)
    want = layers.norm(x, None, None, z, "silu", False, 1e-5, dy)
    dx, dz = torch.empty(T, G, V, device="cuda"), torch.empty(T, G, V, device="cuda")
    gdp.gdp_group_norm_backward(x.cuda(), None, None, z.cuda(), "silu", False, 1e-5, dy.cuda(), dx, None, None, dz, None)
    close(dx, want["dx"], want["dx_bound"], "dx", F32)
    close(dz, want["dgate"], want["dgate_bound"], "dgate", F32)


def test_the_smallest_eps(gdp):  # noqa: F811
    """Groups without variance give the bias, at the smallest eps; groups of tiny values what the formula gives."""
    eps = 2.0 ** -126
    x, w, b, z, dy = make(9, 4, 64, F32, weight="channel", bias=True, gated=False, seed=9)
    flat = torch.full_like(x, 0.5)
    y = gdp.group_norm(flat.cuda(), weight=w.cuda(), bias=b.cuda(), eps=eps)
    assert torch.equal(y.cpu(), b.expand(9, 4, 64))
    d = gdp.group_norm_backward(flat.cuda(), dy.cuda(), weight=w.cuda(), bias=b.cuda(), eps=eps)
    assert all(torch.isfinite(t).all() for t in d.values() if t is not None) and not d["dweight"].any()
    check_norm(gdp, 1e-15 * x, w, b, None, dy, "silu", True, eps=eps)
