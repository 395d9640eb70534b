"""The short causal convolution, its single-token step and its gradients through the binding against the float64 oracle
(needs a gfx950 GPU)."""
import pytest
import torch

from oracle import blocks

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def gdp():
    from gated_deltaproduct_recurrence_amd import binding
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return binding


def dev(t):
    return None if t is None else t.cuda()


def close(got, value, bound, what, dtype):
    got = got.detach().cpu().to(torch.float64)
    limit = blocks.rounded(value, bound, dtype)
    bad = ~((got - value).abs() <= limit)
    assert not bad.any(), (what, int(bad.sum()), tuple(torch.nonzero(bad)[0].tolist()), float(got[bad][0]),
                           float(value[bad][0]), float(limit[bad][0]))


def edges(lens, start=0):
    cu = [start]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def make(lens, D, W, dtype, bias=True, initial=True, wdtype=F32, seed=0, start=0, extra=0):
    gen = torch.Generator().manual_seed(seed)
    cu, N = edges(lens, start), len(lens)
    T = cu[-1] + extra
    d = dict(x=torch.randn(T, D, generator=gen).to(dtype), w=(torch.randn(D, W, generator=gen) * 0.5).to(wdtype), cu=cu,
             b=(torch.randn(D, generator=gen) * 0.3).to(wdtype) if bias else None,
             s0=torch.randn(N, W - 1, D, generator=gen).to(dtype) if initial else None,
             dy=torch.randn(T, D, generator=gen).to(dtype), df=torch.randn(N, W - 1, D, generator=gen))
    return d


def check(gdp, d, act, x=None, dy=None, cu_type=torch.int32, grad_final=True):
    cu = torch.tensor(d["cu"], dtype=cu_type, device="cuda")
    T, D = d["x"].shape
    lo, hi = d["cu"][0], d["cu"][-1]
    want = blocks.conv(d["x"], d["w"], d["cu"], d["b"], act, d["s0"], d["dy"], d["df"] if grad_final else None)
    x = dev(d["x"]) if x is None else x
    form = dict(bias=dev(d["b"]), activation=act, initial_state=dev(d["s0"]))
    out = torch.full((T, D), 7.0, dtype=d["x"].dtype, device="cuda")
    y, fs = gdp.short_conv(x, dev(d["w"]), cu, output_final_state=True, out=out, **form)
    assert y is out and (y[:lo] == 7).all() and (y[hi:] == 7).all()
    close(y[lo:hi], want["y"][lo:hi], want["y_bound"][lo:hi], "y", d["x"].dtype)
    assert torch.equal(fs.cpu().double(), want["final"])
    g = gdp.short_conv_backward(x, dev(d["w"]), cu, dev(d["dy"]) if dy is None else dy,
                                d_final_state=dev(d["df"]) if grad_final else None, **form)
    close(g["dx"], want["dx"], want["dx_bound"], "dx", d["x"].dtype)
    assert (g["dx"][:lo] == 0).all() and (g["dx"][hi:] == 0).all()
    close(g["dweight"], want["dweight"], want["dweight_bound"], "dweight", F32)
    for name, key, given in (("dbias", "dbias", d["b"]), ("d_initial_state", "ds0", d["s0"])):
        if given is None:
            assert g[name] is None
        else:
            close(g[name], want[key], want[key + "_bound"], name, F32)
    return y, fs, g


@pytest.mark.parametrize("W", [2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_taps_and_types(gdp, W, dtype):
    """Sequences shorter than, as long as and longer than the taps, empty ones between."""
    lens = [1, 0, W - 1, W, W + 1, 2, 0, 15, 16, 17, 64, 65, 33]
    check(gdp, make(lens, 70, W, dtype, seed=W), "silu")


@pytest.mark.parametrize("D", [1, 2, 3, 7, 8, 64, 255, 256, 257, 511, 512, 513, 1001, 2048])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_channel_counts(gdp, D, dtype):
    check(gdp, make([5, 40, 1, 90], D, 4, dtype, seed=D), "silu")


@pytest.mark.parametrize("act", [None, "none", "silu", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("initial", [False, True])
@pytest.mark.parametrize("wdtype", [F32, BF16])
def test_forms(gdp, act, bias, initial, wdtype):
    check(gdp, make([3, 100, 0, 29], 96, 4, BF16, bias=bias, initial=initial, wdtype=wdtype, seed=4), act,
          grad_final=initial)


@pytest.mark.parametrize("lens", [[1], [0], [], [0, 0], [4096], [1] * 300, [2000, 1, 1999]])
def test_sequence_counts(gdp, lens):
    check(gdp, make(lens, 64, 4, F32, seed=5), "silu", cu_type=torch.int64)


def test_many_sequences(gdp):
    """More sequences than one and than two steps of 64 tell apart."""
    gen = torch.Generator().manual_seed(6)
    for N in (64, 65, 4096, 5000):
        check(gdp, make(torch.randint(0, 4, (N,), generator=gen).tolist(), 8, 3, F32, seed=7), None)


def test_rows_outside_the_sequences(gdp):
    check(gdp, make([20, 0, 30], 40, 4, BF16, seed=8, start=11, extra=200), "silu")


def test_rows_without_any_sequence(gdp):
    check(gdp, make([], 40, 4, BF16, seed=18, extra=300), "silu")
    check(gdp, make([0, 0], 40, 4, BF16, seed=18, start=30, extra=300), "silu")


def test_long_chunks(gdp):
    """Enough rows and channels for the longest chunks."""
    d = make([700, 1, 0, 12000, 3586], 2056, 4, BF16, seed=9)
    check(gdp, d, "silu")


def test_strides(gdp):
    """x and d_y as slices of wider buffers that start anywhere, outputs in wider ones, a broadcast gradient."""
    d = make([9, 70, 33], 72, 4, BF16, seed=10)
    T, D = d["x"].shape
    wide = torch.zeros(T, 201, dtype=BF16, device="cuda")
    wide[:, 3:3 + D], wide[:, 101:101 + D] = d["x"].cuda(), d["dy"].cuda()
    check(gdp, d, "silu", x=wide[:, 3:3 + D], dy=wide[:, 101:101 + D])
    out = torch.full((T, 150), 5.0, dtype=BF16, device="cuda")
    cu = torch.tensor(d["cu"], device="cuda")
    y, _ = gdp.short_conv(d["x"].cuda(), d["w"].cuda(), cu, bias=d["b"].cuda(), out=out[:, 50:50 + D])
    want = blocks.conv(d["x"], d["w"], d["cu"], d["b"])
    close(y, want["y"], want["y_bound"], "y", BF16)
    assert (out[:, :50] == 5).all() and (out[:, 50 + D:] == 5).all()
    d["dy"] = d["dy"][:1].expand(T, D)
    check(gdp, d, "silu", dy=d["dy"][:1].cuda().expand(T, D))


def test_state_cache(gdp):
    """Final states into slots; indices outside the cache write nothing; the chunks of a prompt one after another give
    what the whole prompt gives, and so does the single-token step."""
    lens, D, W = [5, 2, 0, 40, 3], 48, 4
    d = make(lens, D, W, F16, seed=11)
    cu = torch.tensor(d["cu"], dtype=torch.int32, device="cuda")
    for index in (torch.int32, torch.int64):
        cache = torch.full((6, W - 1, D), 9.0, dtype=F16, device="cuda")
        slots = torch.tensor([4, -1, 0, 6, 2], dtype=index, device="cuda")
        form = dict(bias=dev(d["b"]), activation="silu", initial_state=dev(d["s0"]))
        y, fs = gdp.short_conv(dev(d["x"]), dev(d["w"]), cu, output_final_state=True, state_cache=cache,
                               state_indices=slots, **form)
        for slot, i in ((4, 0), (0, 2), (2, 4)):
            assert torch.equal(cache[slot], fs[i])
        assert (cache[[1, 3, 5]] == 9).all()
    # token by token from the initial states, every sequence at its own pace
    cache = dev(d["s0"]).clone()
    for t in range(max(lens)):
        live = [i for i, n in enumerate(lens) if n > t]
        rows = torch.tensor([d["cu"][i] + t for i in live] + [0], device="cuda")
        step = gdp.short_conv_decode(dev(d["x"])[rows], dev(d["w"]), cache,
                                     torch.tensor(live + [-1], device="cuda"), bias=dev(d["b"]), activation="silu")
        assert (step[-1] == 0).all()
        assert torch.equal(step[:-1], y[rows[:-1]])  # the same sums in the same order
    assert torch.equal(cache, fs)


@pytest.mark.parametrize("W", [2, 4, 8])
@pytest.mark.parametrize("dtype,D", [(F32, 130), (BF16, 1025), (F16, 4096)])
def test_step(gdp, W, dtype, D):
    gen = torch.Generator().manual_seed(W)
    N = 9
    x = torch.randn(N, 2 * D, generator=gen).to(dtype)
    w, b = torch.randn(D, W, generator=gen), torch.randn(D, generator=gen)
    cache = torch.randn(12, W - 1, D, generator=gen).to(dtype)
    slots = torch.tensor([3, -1, 11, 0, 12, 5, 7, -5, 1])
    want = blocks.conv_decode(x[:, D:], w, cache, slots, b, "silu")
    cd, out = cache.cuda(), torch.full((N, D + 3), 4.0, dtype=dtype, device="cuda")
    y = gdp.short_conv_decode(x.cuda()[:, D:], w.cuda(), cd, slots.cuda(), bias=b.cuda(), activation="silu",
                              out=out[:, 1:1 + D])
    close(y, want["y"], want["y_bound"], "y", dtype)
    assert torch.equal(cd.cpu().double(), want["cache"]) and (out[:, 0] == 4).all() and (out[:, 1 + D:] == 4).all()
    assert gdp.short_conv_decode(x[:0, D:].cuda(), w.cuda(), cd, slots[:0].cuda()).shape == (0, D)


def test_a_bad_value_stays_in_its_sequence_and_channel(gdp):
    d = make([30, 50, 20], 64, 4, F32, seed=12)
    d["x"][40, 7], d["x"][60, 9] = float("nan"), float("inf")
    cu = torch.tensor(d["cu"], device="cuda")
    form = dict(bias=dev(d["b"]), activation="silu", initial_state=dev(d["s0"]))
    y, fs = gdp.short_conv(dev(d["x"]), dev(d["w"]), cu, output_final_state=True, **form)
    g = gdp.short_conv_backward(dev(d["x"]), dev(d["w"]), cu, dev(d["dy"]), d_final_state=dev(d["df"]), **form)
    fine = torch.ones(100, 64, dtype=torch.bool)
    fine[40:44, 7] = fine[60:64, 9] = False
    assert torch.isfinite(y.cpu()[fine]).all() and torch.isnan(y.cpu()[40:44, 7]).all()
    fine[37:44, 7] = fine[57:64, 9] = False
    assert torch.isfinite(g["dx"].cpu()[fine]).all()
    channels = torch.ones(64, dtype=torch.bool)
    channels[[7, 9]] = False
    assert torch.isfinite(g["dweight"].cpu()[channels]).all() and torch.isfinite(g["dbias"].cpu()[channels]).all()


def test_far_activations(gdp):
    d = make([50], 32, 4, F32, seed=13)
    d["x"] *= 80.0
    for act in ("silu", "sigmoid"):
        check(gdp, d, act)


def test_streams_graphs_and_repeats(gdp):
    """The same bits again, on another stream, and from a captured graph on new inputs."""
    d = make([100, 7, 0, 300], 520, 4, BF16, seed=14)
    cu = torch.tensor(d["cu"], dtype=torch.int32, device="cuda")
    x, w, b, s0, dy, df = (dev(d[k]) for k in ("x", "w", "b", "s0", "dy", "df"))

    def both():
        y, fs = gdp.short_conv(x, w, cu, bias=b, activation="silu", initial_state=s0, output_final_state=True)
        g = gdp.short_conv_backward(x, w, cu, dy, bias=b, activation="silu", initial_state=s0, d_final_state=df)
        return [y, fs, *g.values()]

    first = both()
    assert all(torch.equal(p, q) for p, q in zip(first, both()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = both()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for seed in (15, 16, 17):
        new = make([100, 7, 0, 300], 520, 4, BF16, seed=seed)
        x.copy_(new["x"]), dy.copy_(new["dy"]), s0.copy_(new["s0"])
        eager = both()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(held, eager))
