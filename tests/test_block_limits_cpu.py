"""Sizes past what the entries serve are refused, whatever they are modulo 2^32: host-side checks, no GPU.  Pointers are
fake, never dereferenced."""
import ctypes

import pytest

from tests import test_abi_cpu as prefill_abi
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


def prefill_backward(b, a):
    r = ctypes.byref
    f, F32 = a["fake"], b.GDP_F32
    shape = lambda t: [t.shape[i] for i in range(t.ndim)]  # noqa: E731
    grads = [f.tensor(b, F32, shape(a[k])) for k in ("q", "k", "v", "g_log", "beta", "s0")]
    return b.LIB.gdp_chunk_prefill_backward(r(a["q"]), r(a["k"]), r(a["v"]), r(a["g_log"]), r(a["beta"]), a["n"], r(a["cu"]),
                                            a["scale"], r(a["s0"]), a["l2"], r(a["o"]), r(b.gdp_tensor()),
                                            *[r(g) for g in grads], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("K,V", [((1 << 32) + 64, 64), (64, (1 << 32) + 64), ((1 << 33) + 128, 128)])
def test_head_sizes_past_32_bits(b, K, V):  # noqa: F811
    """2^32 + 64 is not 64."""
    sizes = dict(Hqk=1, Hv=1, n=1, K=K, V=V)
    prefill_abi.expect(b, prefill_abi.base_args(b, T=3, **sizes), b.GDP_EUNSUPPORTED, "are not served")
    prefill_abi.decode_expect(b, prefill_abi.decode_args(b, N=3, **sizes), b.GDP_EUNSUPPORTED, "are not served")
    a = prefill_abi.base_args(b, T=3, **sizes)
    assert prefill_backward(b, a) == b.GDP_EUNSUPPORTED and "backward needs K, V" in b.gdp_last_error()


def test_head_counts_past_32_bits(b):  # noqa: F811
    a = prefill_abi.base_args(b, T=3, Hqk=1, Hv=(1 << 32) + 4, n=1, K=64, V=64)
    assert prefill_backward(b, a) == b.GDP_EINVAL and "too many sequences or heads" in b.gdp_last_error()
