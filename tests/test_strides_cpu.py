"""A dimension of one element has no stride that matters: torch calls any tensor with one contiguous, and its
contiguous() returns it as it is (host-side, no GPU; pointers are fake, every call is refused for an overlap)."""
import pytest
import torch

from tests.test_abi_cpu import Fake
from tests.test_layer_abi_cpu import change, decode, norm, norm_args, norm_backward, refused, scan, scan_args


@pytest.fixture(scope="module")
def b():
    from gated_deltaproduct_recurrence_amd import binding
    return binding


def test_torch_keeps_such_strides():
    one = torch.zeros(4, 7, dtype=torch.int32)[:1, 3]
    assert one.contiguous().stride() == (7,)
    assert torch.zeros(1, 5).t().contiguous().stride() == (1, 5)


def test_one_cache_slot_out_of_a_table(b):
    f = Fake()
    a = dict(x=f.tensor(b, b.GDP_BF16, [1, 96]), g=f.tensor(b, b.GDP_F32, [1, 96]), comp=0,
             cache=f.tensor(b, b.GDP_F32, [9, 96]), slots=f.tensor(b, b.GDP_I64, [1], [7]),
             o=f.tensor(b, b.GDP_BF16, [1, 96]), fake=f)
    a["o"].data = a["x"].data
    refused(b, decode, a, b.GDP_EALIAS, "o overlaps input x")
    a = change(b, scan_args(b, N=1), slots=(b.GDP_I32, [1], [5]))
    a["o"].data = a["x"].data
    refused(b, scan, a, b.GDP_EALIAS, "o overlaps input x")


def test_one_channel(b):
    a = change(b, scan_args(b, T=200, N=3, D=1), x=(b.GDP_BF16, [200, 1], [1, 200]), g=(b.GDP_F32, [200, 1], [3, 9]))
    a["o"].data = a["x"].data
    refused(b, scan, a, b.GDP_EALIAS, "o overlaps input x")
    for call in (norm, norm_backward):
        a = change(b, norm_args(b, V=1), x=(b.GDP_BF16, [20, 4, 1], [4, 1, 80]), w=(b.GDP_F32, [1], [3]))
        a["y"].data = a["dx"].data = a["x"].data
        refused(b, call, a, b.GDP_EALIAS, "overlaps input x")


def test_no_sequences(b):
    a = change(b, scan_args(b), cu=(b.GDP_I32, [1], [4]), s0=(b.GDP_F32, [0, 96]), fs=(b.GDP_F32, [0, 96]),
               slots=(b.GDP_I32, [0]))
    a["o"].data = a["x"].data
    refused(b, scan, a, b.GDP_EALIAS, "o overlaps input x")
