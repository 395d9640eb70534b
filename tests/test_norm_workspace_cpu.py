"""The workspace of the group norm's gradients: asked for where there are sums to form, and in proportion to the
input (host-side, no GPU; pointers are fake and never dereferenced)."""
import random

import pytest

from tests.test_layer_abi_cpu import change, norm_args, norm_backward, refused


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
