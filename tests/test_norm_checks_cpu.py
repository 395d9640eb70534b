"""Host-side checks of the group norm: eps, and the workspace of the gradients, asked for where there are sums to
form and in proportion to the input (no GPU; pointers are fake and never dereferenced)."""
import random

import pytest

from tests.test_layer_abi_cpu import change, norm, norm_args, norm_backward, refused


@pytest.fixture(scope="module")
def b():
    from gated_deltaproduct_recurrence_amd import binding
    return binding


def test_no_parameters_need_no_workspace(b):
    """Without weight and bias the call is checked past its workspace, to the overlap that it is refused for."""
    for given in (None, "unaligned"):
        a = change(b, norm_args(b), w=None, bias=None, dw=None, db=None)
        a["ws"], a["wsb"] = (None, 0) if given is None else (a["ws"] + 8, 8)
        a["dx"].data = a["x"].data
        refused(b, norm_backward, a, b.GDP_EALIAS, "dx overlaps input x")
    for absent in (dict(w=None, dw=None), dict(bias=None, db=None)):
        a = change(b, norm_args(b), **absent)
        a["ws"], a["wsb"] = None, 0
        refused(b, norm_backward, a, b.GDP_EWORKSPACE, "needed")


def test_the_workspace_follows_the_input(b):
    """At most one row of sums (weight and bias, float32) per group of a token, or per team of a workgroup."""
    need = b.gdp_group_norm_backward_workspace_bytes
    assert need(1, 65535, 8) < 5 << 20 and need(1, 4097, 128) < 5 << 20
    rng = random.Random(7)
    sizes = [(1, 1, 1), (1, 65535, 1), (1, 65535, 16384), (3, 4099, 100), (5, 4097, 16384)]
    for _ in range(3000):
        V = rng.choice([rng.randint(1, 16384), 1 << rng.randint(0, 14)])
        sizes.append((int(2 ** rng.uniform(0, 17)), int(2 ** rng.uniform(0, 15.99)), V))
    for T, G, V in sizes:
        assert 0 < need(T, G, V) <= 8 * V * (T * G + 256) + 255, (T, G, V)


@pytest.mark.parametrize("call", [norm, norm_backward])
def test_eps_below_the_normal_numbers_is_refused(b, call):
    """1 / sqrt serves no subnormal variance; the smallest normal eps is let through, to the overlap."""
    for eps, code, text in ((2.0 ** -127, b.GDP_EINVAL, "eps"), (1e-40, b.GDP_EINVAL, "eps"),
                            (2.0 ** -126, b.GDP_EALIAS, "overlaps input x")):
        a = norm_args(b)
        a["eps"] = eps
        a["y"].data = a["dx"].data = a["x"].data
        refused(b, call, a, code, text)
