"""The oracle's error bounds count the additions of the library's chunks: their lengths, as the workspaces tell them (no
GPU)."""
import itertools

import pytest

from oracle import blocks


@pytest.fixture(scope="module")
def b():
    from gated_deltaproduct_recurrence_amd import binding
    return binding


def round256(x):
    return (x + 255) // 256 * 256


@pytest.mark.parametrize("D", [1, 64, 65, 1001, 2048, 2056, 4096])
def test_convolution(b, D):
    """Partial sums [chunks, W + 2, D]."""
    for T, N, W in itertools.product((0, 1, 16, 1000, 8245, 16288, 32768, 200000), (1, 5, 300), (2, 4)):
        rows = blocks.conv_chunk_rows(T, D)
        assert b.gdp_short_conv_backward_workspace_bytes(T, N, D, W) == round256((T // rows + N) * (W + 2) * D * 4)


@pytest.mark.parametrize("D,G", [(64, 1), (130, 2), (200, 8), (512, 1), (2048, 1), (2600, 1), (4096, 4)])
def test_selective_scan(b, D, G):
    """States [rows / chunk, S, D] and sums of steps [rows / chunk, D] handed on, and up to 1024 chunks' order; in the
    gradients partial sums [blocks, T, 2, S] and [chunks, S + 2, D] besides."""
    S, size = 16, 4 * D
    for T, N in itertools.product((1, 16, 1000, 8192, 33824, 200000), (1, 4, 68, 2000)):
        forward, back = blocks.select_chunk_rows(T, N, D, G)

        def space(rows):
            full, count = (T - 1) // rows, T // rows + N
            return round256(full * S * size) + round256(full * size) + (round256(count * 4) if count <= 1024 else 0)

        assert b.gdp_selective_scan_workspace_bytes(T, N, D, G, S) == space(forward)
        shares = G * -(-(D // G) // 64) * T * 2 * S * 4
        assert b.gdp_selective_scan_backward_workspace_bytes(T, N, D, G, S, True) == (
            space(back) + round256(shares) + round256((T // back + N) * (S + 2) * size))


def test_norms(b):
    """Partial sums [workgroups, 2, D], or two teams' each."""
    for T, D in itertools.product((1, 100, 8195, 100000), (7, 64, 1000, 4096, 5001, 16384)):
        rows = b.gdp_residual_norm_backward_workspace_bytes(T, D) // (8 * D)
        assert rows <= 2 * blocks.NORM_WORKGROUPS
    assert b.gdp_residual_norm_backward_workspace_bytes(100000, 1024) == 8 * 1024 * blocks.NORM_WORKGROUPS


def test_bounds_of_shorter_chunks_are_not_given():
    import torch
    x, A, B = torch.zeros(5000, 1), -torch.ones(1, 1), torch.zeros(5000, 1, 1)
    with pytest.raises(AssertionError, match="shorter chunks"):
        blocks.select(x, x, A, B, B, [0, 5000], join=7)
