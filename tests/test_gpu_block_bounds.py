"""The short convolution and the selective scan write nothing beside their outputs, their caches and the workspace of the
reported size, whatever cu_seqlens and the slots hold (needs a gfx950 GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
GUARD = 8192  # bytes before and behind


@pytest.fixture(scope="module")
def gdp():
    from gated_deltaproduct_recurrence_amd import binding
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return binding


class Guarded:
    """Buffers between bytes that must stay."""

    def __init__(self):
        self.held = []

    def __call__(self, *shape, dtype=F32):
        size = torch.empty(shape, dtype=dtype, device="meta").numel() * dtype.itemsize
        buf = torch.full((size + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        self.held.append((buf, size))
        return buf[GUARD:GUARD + size].view(dtype).view(shape)

    def check(self):
        for buf, size in self.held:
            assert (buf[:GUARD] == 0xA5).all() and (buf[GUARD + size:] == 0xA5).all(), size


def boundaries(T):
    """Rising ones, those that cover a part, and some that do not rise or lie outside."""
    return [[0, T], [0, T // 3, T // 3, T], [5, 40, 41, T - 7], [0, 50, 20, T], [T, 0, T, 40], [-5, 30, T + 110, 60],
            [T, T - 1, 1, 0], [1 << 40, -1 << 40, 17, 1 << 33], list(range(0, T + 1)), list(range(T, -1, -1))]


@pytest.mark.parametrize("W", [2, 4, 8])
@pytest.mark.parametrize("T,D,dtype", [(90, 24, F32), (333, 1001, BF16)])
def test_convolution(gdp, T, D, dtype, W):
    x, dy = torch.randn(T, D, device="cuda").to(dtype), torch.randn(T, D, device="cuda").to(dtype)
    w, b = torch.randn(D, W, device="cuda"), torch.randn(D, device="cuda")
    for bounds in boundaries(T):
        cu, N = torch.tensor(bounds, device="cuda"), len(bounds) - 1
        new = Guarded()
        slots = torch.tensor([(3, -1, 99, 0)[i % 4] if i < 4 else -2 for i in range(N)], device="cuda")
        s0, df = torch.randn(N, W - 1, D, device="cuda").to(dtype), torch.randn(N, W - 1, D, device="cuda")
        gdp.gdp_short_conv(x, w, b, "silu", cu, s0, True, new(4, W - 1, D, dtype=dtype), slots, new(T, D, dtype=dtype),
                           new(N, W - 1, D, dtype=dtype))
        ws = new(gdp.gdp_short_conv_backward_workspace_bytes(T, N, D, W), dtype=torch.uint8)
        gdp.gdp_short_conv_backward(x, w, b, "silu", cu, s0, dy, df, new(T, D, dtype=dtype), new(D, W), new(D),
                                    new(N, W - 1, D), ws)
        new.check()
    new = Guarded()
    slots = torch.tensor([1 << 40, -1, 3, 4, 0, -1 << 40], device="cuda")
    gdp.gdp_short_conv_decode(x[:6], w, b, None, new(4, W - 1, D, dtype=dtype), slots, new(6, D, dtype=dtype))
    new.check()


@pytest.mark.parametrize("S", [3, 8, 16, 32])
@pytest.mark.parametrize("T,D,G,dtype", [(90, 24, 1, F32), (333, 130, 2, BF16)])
def test_selective_scan(gdp, T, D, G, dtype, S):
    rand = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    u, dt, z, do = (rand(T, D).to(dtype) for _ in range(4))
    A, B, C, skip, bias = -rand(D, S).abs(), rand(T, G, S).to(dtype), rand(T, G, S).to(dtype), rand(D), rand(D)
    for bounds in boundaries(T):
        cu, N = torch.tensor(bounds, device="cuda"), len(bounds) - 1
        new = Guarded()
        slots = torch.tensor([(3, -1, 99, 0)[i % 4] if i < 4 else -2 for i in range(N)], device="cuda")
        s0, df = rand(N, D, S), rand(N, D, S)
        points = new(T // 16 + N, S, D)
        ws = new(gdp.gdp_selective_scan_workspace_bytes(T, N, D, G, S), dtype=torch.uint8)
        gdp.gdp_selective_scan(u, dt, A, B, C, skip, z, bias, True, cu, s0, True, new(4, D, S), slots, True,
                               new(T, D, dtype=dtype), new(N, D, S), points, ws)
        for given in (points, None):
            ws = new(gdp.gdp_selective_scan_backward_workspace_bytes(T, N, D, G, S, given is not None), dtype=torch.uint8)
            gdp.gdp_selective_scan_backward(u, dt, A, B, C, skip, z, bias, True, cu, s0, given, do, df,
                                            new(T, D, dtype=dtype), new(T, D, dtype=dtype), new(D, S),
                                            new(T, G, S, dtype=dtype), new(T, G, S, dtype=dtype), new(D),
                                            new(T, D, dtype=dtype), new(D), new(N, D, S), ws)
        new.check()
    new = Guarded()
    slots = torch.tensor([1 << 40, -1, 3, 4, 0, -1 << 40], device="cuda")
    gdp.gdp_selective_scan_decode(u[:6], dt[:6], A, B[:6], C[:6], skip, z[:6], bias, True, new(4, D, S), slots,
                                  new(6, D, dtype=dtype))
    new.check()


@pytest.mark.parametrize("T,D", [(0, 64), (1, 7), (90, 1001), (700, 4096), (5, 16384)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_norms(gdp, T, D, dtype):
    rand = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    x, dr = rand(T, D), rand(T, D)
    y, z, dn = (rand(T, D).to(dtype) for _ in range(3))
    wa, wb = rand(D), rand(D)
    new = Guarded()
    gdp.gdp_residual_norm(x, y, wa, wb, z, "silu", True, True, 0.5, 1e-5, new(T, D), new(T, D, dtype=dtype))
    ws = new(gdp.gdp_residual_norm_backward_workspace_bytes(T, D), dtype=torch.uint8)
    gdp.gdp_residual_norm_backward(x, y, wa, wb, z, "silu", True, True, 0.5, 1e-5, dr, dn, new(T, D),
                                   new(T, D, dtype=dtype), new(D), new(D), new(T, D, dtype=dtype), ws)
    new.check()
