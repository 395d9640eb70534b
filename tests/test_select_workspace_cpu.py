"""Workspaces of the selective scan: room for what chunks hand on, which the rows bound whatever the number of sequences
(no GPU)."""
import pytest

MIB = 1 << 20


@pytest.fixture(scope="module")
def b():
    from gated_deltaproduct_recurrence_amd import binding
    return binding


@pytest.mark.parametrize("T,N,D", [(8192, 8192, 4096), (32768, 4096, 4096), (4096, 1 << 20, 64), (1, 1 << 20, 64)])
def test_many_short_sequences_ask_for_little(b, T, N, D):
    """Sequences of a row to some rows, or of none, hand nothing on."""
    assert b.gdp_selective_scan_workspace_bytes(T, N, D, 1, 16) <= 64 * MIB


@pytest.mark.parametrize("T,N", [(8192, 8192), (1, 1 << 16)])
def test_of_the_gradients(b, T, N):
    """Beside the partial sums of the parameters' gradients, [chunks, S + 2, D], and those of B's and C's."""
    D, S = 256, 16
    sums, shares = (T // 64 + N) * (S + 2) * D * 4, -(-D // 64) * T * 2 * S * 4
    assert b.gdp_selective_scan_backward_workspace_bytes(T, N, D, 1, S, True) <= sums + shares + 64 * MIB


@pytest.mark.parametrize("D,G,S", [(512, 1, 16), (2048, 1, 16), (70, 1, 3), (4096, 8, 32)])
@pytest.mark.parametrize("T", [0, 1, 15, 16, 17, 100, 4097, 100000])
def test_more_sequences_ask_for_no_more_hand_overs(b, T, D, G, S):
    """The order of up to 1024 chunks aside (4 KiB): chunks only get longer with more sequences."""
    sizes = [b.gdp_selective_scan_workspace_bytes(T, N, D, G, S) for N in (1, 2, 7, 64, 1000, 5000)]
    assert all(s <= sizes[0] + 4096 for s in sizes), sizes
