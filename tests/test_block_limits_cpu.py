"""Sizes past what the short convolution and the selective scan serve are refused, whatever they are modulo 2^32: host-side
checks, no GPU.  Pointers are fake, never dereferenced."""
import pytest

from tests import test_block_abi_cpu as abi
from tests.test_block_abi_cpu import b  # noqa: F401  (the fixture)

CONV = {"short_conv": abi.conv, "short_conv_decode": abi.conv_decode, "short_conv_backward": abi.conv_backward}
SELECT = {"selective_scan": abi.select, "selective_scan_decode": abi.select_decode,
          "selective_scan_backward": abi.select_backward}
PAST = [(1 << 24) + 1, 1 << 31, (1 << 32) - 64, 1 << 32, (1 << 32) + 64]


@pytest.mark.parametrize("entry", [*CONV, *SELECT])
@pytest.mark.parametrize("D", PAST)
def test_channels_past_the_limit(b, entry, D):  # noqa: F811
    a = abi.conv_args(b, T=3, D=D) if entry in CONV else abi.select_args(b, T=3, D=D, G=1)
    abi.refused(b, {**CONV, **SELECT}[entry], a, b.GDP_EUNSUPPORTED, f"more than {1 << 24} channels")


@pytest.mark.parametrize("entry", [*CONV, *SELECT])
def test_few_channels_out_of_very_many(b, entry):  # noqa: F811
    """Inputs of 2^32 + 64 channels, outputs and states of 64."""
    make = abi.conv_args if entry in CONV else lambda b, **new: abi.select_args(b, G=1, **new)
    a, wide = make(b, T=3, D=64), make(b, T=3, D=(1 << 32) + 64)
    for k in ("x", "w", "bc", "u", "dt", "A", "skip", "z", "bias"):
        if k in a:
            a[k] = wide[k]
    abi.refused(b, {**CONV, **SELECT}[entry], a, b.GDP_EUNSUPPORTED, f"more than {1 << 24} channels")


def test_workspaces_of_sizes_past_the_limits(b):  # noqa: F811
    for D in PAST:
        assert b.gdp_short_conv_backward_workspace_bytes(3, 3, D, 4) == 0
        assert b.gdp_selective_scan_workspace_bytes(3, 3, D, 1, 16) == 0
        assert b.gdp_selective_scan_backward_workspace_bytes(3, 3, D, 1, 16, True) == 0
