"""The selective state space scan, its single-token step and its gradients through the binding against the float64
oracle (needs a gfx950 GPU)."""
import pytest
import torch

from oracle import blocks
from tests.test_gpu_short_conv import close, dev, edges

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
GRADS = ("du", "ddt", "dA", "dB", "dC", "dskip", "dgate", "ddt_bias", "ds0")


@pytest.fixture(scope="module")
def gdp():
    from gated_deltaproduct_recurrence_amd import binding
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return binding


def make(lens, D, S, dtype, dt_type=None, G=1, gated=True, skip=True, bias=True, initial=True, softplus=True, seed=0,
         start=0, extra=0):
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    cu, N = edges(lens, start), len(lens)
    T = cu[-1] + extra
    dt = rand(T, D) if softplus else rand(T, D).abs() * 0.1
    return dict(u=rand(T, D).to(dtype), dt=dt.to(dt_type or dtype), A=-torch.rand(D, S, generator=gen) * 4 - 0.05,
                B=rand(T, G, S).to(dtype), C=rand(T, G, S).to(dtype), skip=rand(D) if skip else None,
                z=rand(T, D).to(dtype) if gated else None, bias=rand(D).abs() * 0.1 - (2 if softplus else 0) if bias else None,
                softplus=softplus, cu=cu, s0=rand(N, D, S) if initial else None, do=rand(T, D).to(dtype),
                df=rand(N, D, S))


def oracle(d, back=True, **form):
    return blocks.select(d["u"], d["dt"], d["A"], d["B"], d["C"], d["cu"], d["skip"], d["z"], d["bias"], d["softplus"],
                         d["s0"], d["do"] if back else None, d["df"] if back else None, **form)


def on_gpu(d, cu_type=torch.int32):
    on = {k: dev(v) for k, v in d.items() if isinstance(v, torch.Tensor) or v is None}
    on["cu"] = torch.tensor(d["cu"], dtype=cu_type, device="cuda")
    return on


def form_of(on, d):
    return dict(skip=on["skip"], gate=on["z"], dt_bias=on["bias"], dt_softplus=d["softplus"], initial_state=on["s0"])


def compare(d, want, g):
    types = dict(du=d["u"].dtype, dgate=d["u"].dtype, dB=d["u"].dtype, dC=d["u"].dtype, ddt=d["dt"].dtype)
    given = dict(dskip=d["skip"], dgate=d["z"], ddt_bias=d["bias"], ds0=d["s0"])
    for name in GRADS:
        got = g["d_initial_state" if name == "ds0" else name]
        if name in given and given[name] is None:
            assert got is None
        else:
            close(got, want[name], want[name + "_bound"], name, types.get(name, F32))


def check(gdp, d, on=None, cu_type=torch.int32, **bounds):
    on = on or on_gpu(d, cu_type)
    T, D = d["u"].shape
    lo, hi = d["cu"][0], d["cu"][-1]
    want = oracle(d, **bounds)
    args, form = (on["u"], on["dt"], on["A"], on["B"], on["C"], on["cu"]), form_of(on, d)
    out = torch.full((T, D), 7.0, dtype=d["u"].dtype, device="cuda")
    o, fs, points = gdp.selective_scan(*args, output_final_state=True, return_checkpoints=True, out=out, **form)
    assert o is out and (o[:lo] == 7).all() and (o[hi:] == 7).all()
    close(o[lo:hi], want["o"][lo:hi], want["o_bound"][lo:hi], "o", d["u"].dtype)
    close(fs, want["final"], want["final_bound"], "final", F32)
    g = gdp.selective_scan_backward(*args, on["do"], d_final_state=on["df"], checkpoints=points, **form)
    compare(d, want, g)
    again = gdp.selective_scan_backward(*args, on["do"], d_final_state=on["df"], **form)
    for name, t in g.items():
        assert (t is None) == (again[name] is None) and (t is None or torch.equal(t, again[name])), name
    return o, fs, g


@pytest.mark.parametrize("S", [1, 2, 3, 4, 5, 7, 8, 12, 16, 17, 31, 32])
def test_state_counts(gdp, S):
    check(gdp, make([1, 15, 0, 16, 17, 40, 100], 70, S, F32, seed=S))


@pytest.mark.parametrize("dtype,dt_type", [(F32, F32), (BF16, F32), (BF16, BF16), (F16, F32), (F16, F16)])
@pytest.mark.parametrize("S", [3, 16])
def test_types(gdp, dtype, dt_type, S):
    check(gdp, make([33, 1, 64, 0, 31], 96, S, dtype, dt_type, seed=1))


@pytest.mark.parametrize("D,G", [(1, 1), (3, 3), (63, 1), (64, 1), (65, 1), (128, 2), (130, 2), (200, 8), (257, 1), (512, 4)])
def test_channels_and_groups(gdp, D, G):
    check(gdp, make([5, 40, 1, 30], D, 8, F32, G=G, seed=D))


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("skip,bias", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("initial", [False, True])
@pytest.mark.parametrize("softplus", [False, True])
def test_forms(gdp, gated, skip, bias, initial, softplus):
    check(gdp, make([3, 50, 0, 29], 72, 16, F32, gated=gated, skip=skip, bias=bias, initial=initial, softplus=softplus,
                    seed=2))


@pytest.mark.parametrize("lens", [[1], [0], [], [0, 0], [2], [16], [31], [32], [33], [64], [65], [400], [1] * 100, [300, 1, 299]])
def test_sequence_counts(gdp, lens):
    """One to many chunks per sequence, in both directions."""
    check(gdp, make(lens, 40, 6, F32, seed=3), cu_type=torch.int64)


def test_many_sequences(gdp):
    gen = torch.Generator().manual_seed(4)
    for N in (64, 65, 4100):
        check(gdp, make(torch.randint(0, 3, (N,), generator=gen).tolist(), 8, 2, F32, seed=5))


def test_rows_outside_the_sequences(gdp):
    check(gdp, make([20, 0, 90], 40, 16, BF16, F32, seed=6, start=11, extra=70))


def test_rows_without_any_sequence(gdp):
    check(gdp, make([], 40, 16, BF16, F32, seed=19, extra=300))
    check(gdp, make([0, 0], 40, 16, BF16, F32, seed=19, start=30, extra=300))


@pytest.mark.parametrize("D", [1280, 2600])
def test_uneven_sequences_in_their_order_of_length(gdp, D):
    """Enough waves and sequences for the long chunks to be taken first, of many lengths, empty ones among them."""
    gen = torch.Generator().manual_seed(20)
    lens = torch.randint(0, 90, (60,), generator=gen).tolist() + [0, 700, 1, 0]
    check(gdp, make(lens, D, 2, F32, seed=20))


def test_one_long_sequence(gdp):
    """More chunks than the walks over them read ahead."""
    check(gdp, make([1500], 20, 4, F32, seed=7))


def test_long_chunks(gdp):
    """Chunks of 2048 rows on the way forward and back, against the oracle in a few channels.  B and C are shared by all
    channels, whose dB and dC the oracle does not form."""
    lens, D, S = [4500, 3, 0, 2048, 2049] + [4096] * 30, 4096, 4
    gen = torch.Generator(device="cuda").manual_seed(8)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    cu = edges(lens)
    T, N = cu[-1], len(lens)
    on = dict(u=rand(T, D).to(BF16), dt=rand(T, D).to(BF16), A=-torch.rand(D, S, generator=gen, device="cuda") * 2 - 0.05,
              B=rand(T, 1, S).to(BF16), C=rand(T, 1, S).to(BF16), skip=rand(D), z=None, bias=rand(D) * 0.1 - 4,
              cu=torch.tensor(cu, device="cuda"), s0=rand(N, D, S), do=rand(T, D).to(BF16), df=rand(N, D, S))
    d = dict(softplus=True)
    args, form = (on["u"], on["dt"], on["A"], on["B"], on["C"], on["cu"]), form_of(on, d)
    o, fs, points = gdp.selective_scan(*args, output_final_state=True, return_checkpoints=True, **form)
    g = gdp.selective_scan_backward(*args, on["do"], d_final_state=on["df"], checkpoints=points, **form)
    for ch in (0, 777, 4095):
        one = slice(ch, ch + 1)
        part = dict(u=on["u"][:, one], dt=on["dt"][:, one], A=on["A"][one], B=on["B"], C=on["C"], skip=on["skip"][one],
                    z=None, bias=on["bias"][one], softplus=True, cu=cu, s0=on["s0"][:, one], do=on["do"][:, one],
                    df=on["df"][:, one])
        want = oracle(part, join=600, chain=2048)
        close(o[:, one], want["o"], want["o_bound"], "o", BF16)
        close(fs[:, one], want["final"], want["final_bound"], "final", F32)
        for name, got, dtype in (("du", g["du"][:, one], BF16), ("ddt", g["ddt"][:, one], BF16), ("dA", g["dA"][one], F32),
                                 ("dskip", g["dskip"][one], F32), ("ddt_bias", g["ddt_bias"][one], F32),
                                 ("ds0", g["d_initial_state"][:, one], F32)):
            close(got, want[name], want[name + "_bound"], name, dtype)


def test_strides(gdp):
    """Operands as slices of one wide projection that start anywhere, groups that are not neighbours, wide outputs."""
    d = make([9, 70, 33], 72, 5, BF16, G=2, seed=9)
    on = on_gpu(d)
    T, D = d["u"].shape
    wide = torch.zeros(T, 400, dtype=BF16, device="cuda")
    at = 1
    for k in ("u", "dt", "z", "do"):
        wide[:, at:at + D] = on[k]
        on[k] = wide[:, at:at + D]
        at += D + 3
    for k in ("B", "C"):
        wide[:, at:at + 28].view(T, 2, 14)[:, :, 1:6] = on[k]
        on[k] = wide[:, at:at + 28].view(T, 2, 14)[:, :, 1:6]
        at += 29
    check(gdp, d, on)
    d["do"] = d["do"][:1].expand(T, D)
    on["do"] = on["do"][:1].expand(T, D)
    check(gdp, d, on)


def test_gradients_into_wide_buffers(gdp):
    d = make([9, 40], 30, 6, F32, seed=10, extra=5)
    on = on_gpu(d)
    T, D = d["u"].shape
    N, S = 2, 6
    want = oracle(d)
    held = {k: torch.full((T, 50), 3.0, device="cuda") for k in ("du", "ddt", "dgate")}
    view = {k: t[:, 7:7 + D] for k, t in held.items()}
    dA, dB, dC = torch.empty(D, S, device="cuda"), torch.empty(T, 1, S, device="cuda"), torch.empty(T, 1, S, device="cuda")
    dk, db, ds = torch.empty(D, device="cuda"), torch.empty(D, device="cuda"), torch.empty(N, D, S, device="cuda")
    ws = torch.empty(gdp.gdp_selective_scan_backward_workspace_bytes(T, N, D, 1, S, False), dtype=torch.uint8, device="cuda")
    gdp.gdp_selective_scan_backward(on["u"], on["dt"], on["A"], on["B"], on["C"], on["skip"], on["z"], on["bias"], True,
                                    on["cu"], on["s0"], None, on["do"], on["df"], view["du"], view["ddt"], dA, dB, dC, dk,
                                    view["dgate"], db, ds, ws)
    compare(d, want, dict(view, dA=dA, dB=dB, dC=dC, dskip=dk, ddt_bias=db, d_initial_state=ds))
    for t in held.values():
        assert (t[:, :7] == 3).all() and (t[:, 7 + D:] == 3).all()


def test_state_cache_and_steps(gdp):
    """Final states into slots; and the prompt token by token through the single-token step."""
    lens = [5, 2, 0, 40, 3]
    d = make(lens, 48, 16, F16, F32, seed=11)
    on = on_gpu(d)
    want = oracle(d, back=False)
    for index in (torch.int32, torch.int64):
        cache = torch.full((6, 48, 16), 9.0, device="cuda")
        slots = torch.tensor([4, -1, 0, 6, 2], dtype=index, device="cuda")
        o, fs = gdp.selective_scan(on["u"], on["dt"], on["A"], on["B"], on["C"], on["cu"], output_final_state=True,
                                   state_cache=cache, state_indices=slots, **form_of(on, d))
        for slot, i in ((4, 0), (0, 2), (2, 4)):
            assert torch.equal(cache[slot], fs[i])
        assert (cache[[1, 3, 5]] == 9).all()
    cache = on["s0"].clone()
    form = {k: v for k, v in form_of(on, d).items() if k not in ("initial_state", "gate")}
    for t in range(max(lens)):
        live = [i for i, n in enumerate(lens) if n > t]
        rows = torch.tensor([d["cu"][i] + t for i in live] + [0], device="cuda")
        step = gdp.selective_scan_decode(on["u"][rows], on["dt"][rows], on["A"], on["B"][rows], on["C"][rows], cache,
                                         torch.tensor(live + [-1], device="cuda"), gate=on["z"][rows], **form)
        assert (step[-1] == 0).all()
        at = rows[:-1].cpu()
        close(step[:-1], want["o"][at], want["o_bound"][at], "o", F16)
    close(cache, want["final"], want["final_bound"], "cache", F32)


@pytest.mark.parametrize("S", [1, 3, 4, 8, 13, 16, 32])
@pytest.mark.parametrize("dtype,dt_type,D,G", [(F32, F32, 130, 2), (BF16, BF16, 1025, 1), (F16, F32, 512, 8)])
def test_step(gdp, S, dtype, dt_type, D, G):
    N = 9
    d = make([1] * N, D, S, dtype, dt_type, G=G, seed=S)
    on = on_gpu(d)
    gen = torch.Generator().manual_seed(S)
    cache, slots = torch.randn(12, D, S, generator=gen), torch.tensor([3, -1, 11, 0, 12, 5, 7, -5, 1])
    want = blocks.select_decode(d["u"], d["dt"], d["A"], d["B"], d["C"], cache, slots, skip=d["skip"], gate=d["z"],
                                dt_bias=d["bias"], dt_softplus=True)
    cd, out = cache.cuda(), torch.full((N, D + 3), 4.0, dtype=dtype, device="cuda")
    o = gdp.selective_scan_decode(on["u"], on["dt"], on["A"], on["B"], on["C"], cd, slots.cuda(), skip=on["skip"],
                                  gate=on["z"], dt_bias=on["bias"], dt_softplus=True, out=out[:, 1:1 + D])
    close(o, want["o"], want["o_bound"], "o", dtype)
    close(cd, want["cache"], want["cache_bound"], "cache", F32)
    untouched = [2, 4, 6, 8, 9, 10]
    assert torch.equal(cd[untouched].cpu(), cache[untouched]) and (out[:, 0] == 4).all() and (out[:, 1 + D:] == 4).all()
    z = lambda k: on[k][:0]  # noqa: E731
    assert gdp.selective_scan_decode(z("u"), z("dt"), on["A"], z("B"), z("C"), cd, slots[:0].cuda()).shape == (0, D)


def test_small_and_large_steps(gdp):
    """Softplus far out on both sides: steps near 0, whose logarithm would lose all digits of 1 + e, and steps that drop
    the state; and no skip or decay at all."""
    d = make([60], 64, 8, F32, seed=12)
    d["dt"][:20], d["dt"][20:40] = d["dt"][:20] - 20, d["dt"][20:40] + 30
    d["dt"][40:50] = -200.0  # exp underflows: a step of 0
    check(gdp, d)
    d["A"][:, 3] = 0.0
    check(gdp, d)


def test_bad_values_stay_in_their_sequence_and_channel(gdp):
    d = make([30, 50, 20], 64, 16, F32, seed=13)
    d["u"][40, 7], d["dt"][60, 9], d["z"][45, 11] = float("nan"), float("nan"), float("inf")
    on = on_gpu(d)
    args, form = (on["u"], on["dt"], on["A"], on["B"], on["C"], on["cu"]), form_of(on, d)
    o, fs = gdp.selective_scan(*args, output_final_state=True, **form)
    g = gdp.selective_scan_backward(*args, on["do"], d_final_state=on["df"], **form)
    fine = torch.ones(100, 64, dtype=torch.bool)
    fine[40:80, 7] = fine[60:80, 9] = fine[45, 11] = False
    assert torch.isfinite(o.cpu()[fine]).all() and torch.isnan(o.cpu()[40:80, 7]).all()
    assert torch.isfinite(fs.cpu()[[0, 2]]).all() and torch.isfinite(fs.cpu()[1, :7]).all()
    fine[30:80, 7] = fine[30:80, 9] = fine[30:80, 11] = False
    for k in ("du", "ddt", "dgate"):
        assert torch.isfinite(g[k].cpu()[fine]).all()
    others = torch.ones(64, dtype=torch.bool)
    others[[7, 9, 11]] = False
    assert torch.isfinite(g["dA"].cpu()[others]).all() and torch.isfinite(g["dskip"].cpu()[others]).all()
    for k in ("dB", "dC"):  # sums over channels: the other sequences' rows
        assert torch.isfinite(g[k].cpu()[:30]).all() and torch.isfinite(g[k].cpu()[80:]).all()


def test_the_last_row_leaves_no_trace(gdp):
    """An infinite last input reaches the final state, not the gradient of A, which sees the states before rows alone."""
    d = make([5, 21], 64, 4, F32, gated=False, seed=14)
    d["u"][4, 3] = d["u"][25, 5] = float("inf")
    on = on_gpu(d)
    g = gdp.selective_scan_backward(on["u"], on["dt"], on["A"], on["B"], on["C"], on["cu"], on["do"],
                                    d_final_state=on["df"], **form_of(on, d))
    assert torch.isfinite(g["dA"]).all() and torch.isfinite(g["d_initial_state"]).all()


def test_streams_graphs_and_repeats(gdp):
    lens = [300, 7, 0, 190]
    d = make(lens, 200, 16, BF16, seed=15)
    on = on_gpu(d)
    args, form = (on["u"], on["dt"], on["A"], on["B"], on["C"], on["cu"]), form_of(on, d)

    def both():
        o, fs, points = gdp.selective_scan(*args, output_final_state=True, return_checkpoints=True, **form)
        g = gdp.selective_scan_backward(*args, on["do"], d_final_state=on["df"], checkpoints=points, **form)
        return [o, fs, *g.values()]

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
    for seed in (16, 17, 18):
        new = make(lens, 200, 16, BF16, seed=seed)
        for k in ("u", "dt", "B", "C", "z", "s0", "do"):
            on[k].copy_(new[k])
        eager = both()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(held, eager))
