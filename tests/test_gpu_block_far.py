"""Operands that reach far: larger than the memory-side cache (their loads and stores take another path), rows and cache
slots past 32-bit offsets (needs a gfx950 GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def gdp():
    from gated_deltaproduct_recurrence_amd import binding
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return binding


def rand(seed, *shape, dtype=F32):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


@pytest.mark.parametrize("D,shift", [(4096, 0), (4099, 1)])
def test_convolution_of_a_large_stream(gdp, D, shift):
    """The large call's rows against calls on one sequence each, which are small enough for the other path; an odd channel
    count and a stream that starts at an odd element."""
    lens = [9000, 9001, 1, 15998]
    T = sum(lens)
    buf = rand(0, T * D + shift, dtype=BF16)
    x, dy = buf[shift:].view(T, D), rand(1, T, D, dtype=BF16)
    w, b = rand(2, D, 4) * 0.5, rand(3, D)
    assert x.numel() * 4 > 256 << 20
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], device="cuda")
    y, fs = gdp.short_conv(x, w, cu, bias=b, activation="silu", output_final_state=True)
    g = gdp.short_conv_backward(x, w, cu, dy, bias=b, activation="silu")
    for i, n in enumerate(lens):
        lo = int(cu[i])
        one = torch.tensor([0, n], device="cuda")
        part = x[lo:lo + n].clone()
        y1, fs1 = gdp.short_conv(part, w, one, bias=b, activation="silu", output_final_state=True)
        g1 = gdp.short_conv_backward(part, w, one, dy[lo:lo + n], bias=b, activation="silu")
        assert torch.equal(y[lo:lo + n], y1) and torch.equal(fs[i], fs1[0]) and torch.equal(g["dx"][lo:lo + n], g1["dx"])


@pytest.mark.parametrize("D,shift", [(4096, 0), (4099, 1)])
@pytest.mark.parametrize("gated", [False, True])
def test_norms_of_a_large_stream(gdp, D, shift, gated):
    T = 20000
    x, y = rand(4, T * D + shift, dtype=F32)[shift:].view(T, D), rand(5, T * D + shift, dtype=BF16)[shift:].view(T, D)
    z = rand(6, T, D, dtype=BF16) if gated else None
    dr, dn = rand(7, T, D), rand(8, T, D, dtype=BF16)
    form = dict(post_weight=rand(9, D), pre_weight=rand(10, D), activation="silu" if gated else None, residual_scale=0.5)
    r, n = gdp.residual_norm(x, y, gate=z, **form)
    g = gdp.residual_norm_backward(x, y, dr, dn, gate=z, **form)
    for lo, hi in ((0, 700), (9999, 10700), (19300, T)):
        part = lambda t: None if t is None else t[lo:hi].clone()  # noqa: E731
        r1, n1 = gdp.residual_norm(part(x), part(y), gate=part(z), **form)
        g1 = gdp.residual_norm_backward(part(x), part(y), part(dr), part(dn), gate=part(z), **form)
        assert torch.equal(r[lo:hi], r1) and torch.equal(n[lo:hi], n1)
        for k in ("dx", "dy") + (("dgate",) if gated else ()):
            assert torch.equal(g[k][lo:hi], g1[k]), k


def far(t, stride=(1 << 30) + 1):
    """t's rows 2^30 + 1 elements apart."""
    view = torch.empty(t.shape[0] * stride, dtype=t.dtype, device="cuda").as_strided(t.shape, (stride, 1))
    view.copy_(t)
    return view


def test_rows_far_apart(gdp):
    T, D, S = 5, 200, 6
    cu = torch.tensor([0, 2, 5], device="cuda")
    x, d = rand(11, T, D, dtype=BF16), rand(12, T, D, dtype=BF16)
    w = rand(13, D, 3)
    xf, out = far(x), far(torch.zeros_like(x))
    gdp.short_conv(xf, w, cu, out=out)
    assert torch.equal(out, gdp.short_conv(x, w, cu)[0])
    assert torch.equal(gdp.short_conv_backward(xf, w, cu, d)["dx"], gdp.short_conv_backward(x, w, cu, d)["dx"])
    A, B = -rand(14, D, S).abs() - 0.1, rand(15, T, 1, S, dtype=BF16)
    gdp.selective_scan(xf, x, A, B, B, cu, dt_softplus=True, out=out)
    assert torch.equal(out, gdp.selective_scan(x, x, A, B, B, cu, dt_softplus=True)[0])
    a, b = (gdp.selective_scan_backward(t, x, A, B, B, cu, d, dt_softplus=True) for t in (xf, x))
    assert all(torch.equal(a[k], b[k]) for k in ("du", "ddt", "dA", "dB", "dC"))
    gdp.gdp_residual_norm(xf, x, None, None, None, None, True, True, 1.0, 1e-5, out, torch.empty_like(x))
    assert torch.equal(out, gdp.residual_norm(x, x)[0])


def test_cache_slots_far_apart(gdp):
    """Caches of more than 2^32 bytes, their first and last slots in use."""
    N, D, S, W = 3, 4096, 16, 8
    slots = 17000
    index = torch.tensor([slots - 1, -1, 0], device="cuda")
    small = torch.tensor([1, -1, 0], device="cuda")
    x, dt = rand(16, N, D, dtype=BF16), rand(17, N, D, dtype=BF16)
    A, B = -rand(18, D, S).abs() - 0.1, rand(19, N, 1, S, dtype=BF16)
    cu = torch.tensor([0, 1, 2, 3], device="cuda")
    cache = torch.empty(slots, D, S, device="cuda")
    assert cache.numel() * 4 > 1 << 32
    near = rand(20, 2, D, S)
    cache[0], cache[-1] = near[0], near[1]
    o = gdp.selective_scan_decode(x, dt, A, B, B, cache, index, dt_softplus=True)
    assert torch.equal(o, gdp.selective_scan_decode(x, dt, A, B, B, near, small, dt_softplus=True))
    assert torch.equal(cache[0], near[0]) and torch.equal(cache[-1], near[1])
    for c, i in ((cache, index), (near, small)):
        gdp.selective_scan(x, dt, A, B, B, cu, dt_softplus=True, state_cache=c, state_indices=i)
    assert torch.equal(cache[0], near[0]) and torch.equal(cache[-1], near[1])
    slots = 80000
    index[0] = slots - 1
    w = rand(21, D, W)
    cache = torch.empty(slots, W - 1, D, dtype=BF16, device="cuda")
    assert cache.numel() * 2 > 1 << 32
    near = rand(22, 2, W - 1, D, dtype=BF16)
    cache[0], cache[-1] = near[0], near[1]
    y = gdp.short_conv_decode(x, w, cache, index)
    assert torch.equal(y, gdp.short_conv_decode(x, w, near, small))
    assert torch.equal(cache[0], near[0]) and torch.equal(cache[-1], near[1])
    for c, i in ((cache, index), (near, small)):
        gdp.short_conv(x, w, cu, state_cache=c, state_indices=i)
    assert torch.equal(cache[0], near[0]) and torch.equal(cache[-1], near[1])
