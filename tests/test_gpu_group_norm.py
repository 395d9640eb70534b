"""The group norm with an activation and its gradients through the binding against the float64 oracle, and the
layers run together (needs a gfx950 GPU)."""
import pytest
import torch

from oracle import layers

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
    limit = layers.rounded(value, bound, dtype)
    bad = ~((got - value).abs() <= limit)
    assert not bad.any(), (what, int(bad.sum()), tuple(torch.nonzero(bad)[0].tolist()), float(got[bad][0]),
                           float(value[bad][0]), float(limit[bad][0]))


def make(T, G, V, dtype, weight="head", bias=False, gated=True, wdtype=F32, seed=0):
    gen = torch.Generator().manual_seed(seed)
    x, z, dy = ((torch.randn(T, G, V, generator=gen) * s + m).to(dtype) for s, m in ((1.0, 0.3), (2.0, 0.0), (1.0, 0.0)))
    shape = {"head": (V,), "channel": (G, V)}.get(weight)
    w = None if shape is None else (1 + 0.3 * torch.randn(*shape, generator=gen)).to(wdtype)
    b = (0.3 * torch.randn(*(shape or (G, V)), generator=gen)).to(wdtype) if bias else None
    return x, w, b, (z if gated else None), dy


def check_norm(gdp, x, w, b, z, dy, act, center, eps=1e-5, xd=None, zd=None, dyd=None, out=None):
    want = layers.norm(x, w, b, z, act, center, eps, dy)
    form = dict(weight=dev(w), bias=dev(b), gate=dev(z) if zd is None else zd, activation=act, subtract_mean=center,
                eps=eps)
    xd = dev(x) if xd is None else xd
    y = gdp.group_norm(xd, out=out, **form)
    close(y, want["y"], want["y_bound"], "y", x.dtype)
    d = gdp.group_norm_backward(xd, dev(dy) if dyd is None else dyd, **form)
    close(d["dx"], want["dx"], want["dx_bound"], "dx", x.dtype)
    if z is not None:
        close(d["dgate"], want["dgate"], want["dgate_bound"], "dgate", x.dtype)
    for name, p in (("dweight", w), ("dbias", b)):
        if p is None:
            assert d[name] is None
        else:
            close(d[name], want[name], want[name + "_bound"], name, F32)


@pytest.mark.parametrize("V", [1, 2, 7, 16, 24, 64, 77, 96, 100, 128, 256, 500, 512, 513, 1000, 2048])
@pytest.mark.parametrize("G", [1, 3])
def test_group_sizes(gdp, V, G):
    check_norm(gdp, *make(9, G, V, BF16, bias=True, seed=V), "silu", V > 1)


@pytest.mark.parametrize("V", [4096, 5000, 16384])
def test_wide_groups(gdp, V):
    check_norm(gdp, *make(5, 2, V, F32, weight="channel", bias=True, seed=V), "silu", True)
    check_norm(gdp, *make(3, 1, V, BF16, seed=V), "silu", False)


@pytest.mark.parametrize("dtype,wdtype", [(F32, F32), (BF16, F32), (BF16, BF16), (F16, F32), (F16, F16)])
@pytest.mark.parametrize("V", [128, 90])
@pytest.mark.parametrize("weight", ["head", "channel"])
def test_types(gdp, dtype, wdtype, V, weight):
    check_norm(gdp, *make(37, 4, V, dtype, weight=weight, bias=True, wdtype=wdtype, seed=1), "silu", True)


@pytest.mark.parametrize("act", [None, "none", "silu", "sigmoid"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("weight,bias", [("none", False), ("none", True), ("head", False), ("channel", True)])
def test_forms(gdp, act, gated, center, weight, bias):
    check_norm(gdp, *make(21, 5, 64, F32, weight=weight, bias=bias, gated=gated, seed=2), act, center)


@pytest.mark.parametrize("T,G", [(0, 3), (1, 1), (1, 32), (1000, 1), (300, 7), (2, 257), (4099, 2)])
def test_token_and_group_counts(gdp, T, G):
    check_norm(gdp, *make(T, G, 32, F32, weight="channel", bias=True, seed=3), "silu", True)
    check_norm(gdp, *make(T, G, 32, F32, weight="head", bias=True, seed=4), "silu", True)


def test_strided_operands(gdp):
    """x inside a wider projection, a gate whose groups are the outer dimension, an output in a wider buffer."""
    x, w, b, z, dy = make(50, 4, 64, BF16, bias=True, seed=5)
    wide = torch.full((50, 4, 200), 9.0, dtype=BF16, device="cuda")
    wide[:, :, 100:164] = x.cuda()
    zt = z.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.full((50, 8, 64), 9.0, dtype=BF16, device="cuda")
    check_norm(gdp, x, w, b, z, dy, "silu", True, xd=wide[:, :, 100:164], zd=zt, out=out[:, 2:6])
    assert (out[:, :2] == 9).all() and (out[:, 6:] == 9).all()
    odd = torch.empty(50 * 4 * 65 + 1, dtype=BF16, device="cuda")[1:].view(50, 4, 65)
    odd[:, :, :64] = x.cuda()
    check_norm(gdp, x, w, b, z, dy, "silu", False, xd=odd[:, :, :64])
    # a gradient broadcast over the groups
    dyb = dy[:, :1].expand(-1, 4, -1)
    check_norm(gdp, x, w, b, z, dyb, "silu", True, dyd=dy[:, :1].cuda().expand(-1, 4, -1))


@pytest.mark.parametrize("V", [64, 65])
def test_strided_gradients(gdp, V):
    """Gradients written into wider buffers and with the groups as the outer dimension, through the direct call."""
    x, w, b, z, dy = make(30, 3, V, F32, weight="channel", bias=True, seed=17)
    want = layers.norm(x, w, b, z, "sigmoid", True, 1e-5, dy)
    wide = torch.full((30, 3, V + 9), 9.0, device="cuda")
    outer = torch.full((3, 31, V), 9.0, device="cuda")
    dx, dz = wide[:, :, 4:4 + V], outer[:, :30].transpose(0, 1)
    dw, db = torch.empty(3, V, device="cuda"), torch.empty(3, V, device="cuda")
    ws = torch.empty(gdp.gdp_group_norm_backward_workspace_bytes(30, 3, V), dtype=torch.uint8, device="cuda")
    gdp.gdp_group_norm_backward(x.cuda(), w.cuda(), b.cuda(), z.cuda(), "sigmoid", True, 1e-5, dy.cuda(), dx, dw, db, dz, ws)
    for name, got in (("dx", dx), ("dgate", dz), ("dweight", dw), ("dbias", db)):
        close(got, want[name], want[name + "_bound"], name, F32)
    assert (wide[:, :, :4] == 9).all() and (wide[:, :, 4 + V:] == 9).all() and (outer[:, 30] == 9).all()


def test_large_means_and_flat_groups(gdp):
    """A mean far above the spread (two passes over the values), and groups of equal values."""
    x, w, b, z, dy = make(16, 2, 256, F32, bias=True, seed=6)
    check_norm(gdp, x + 1000.0, w, b, z, dy, "silu", True)
    x[3], x[5, 1] = 2.5, 0.0
    check_norm(gdp, x, w, b, z, dy, "silu", True)
    check_norm(gdp, x, w, b, z, dy, "sigmoid", False)


def test_far_activations(gdp):
    """Gates far out on both sides: no overflow on the way."""
    x, w, b, z, dy = make(8, 2, 64, F32, seed=7)
    z = z * 60.0
    for act in ("silu", "sigmoid"):
        check_norm(gdp, x, w, b, z, dy, act, True)


def test_a_bad_value_stays_in_its_group(gdp):
    x, w, b, z, dy = make(40, 4, 128, F32, bias=True, seed=8)
    x[7, 2, 5], x[30, 1, 0] = float("nan"), float("inf")
    y = gdp.group_norm(x.cuda(), w.cuda(), b.cuda(), z.cuda(), "silu")
    d = gdp.group_norm_backward(x.cuda(), dy.cuda(), w.cuda(), b.cuda(), z.cuda(), "silu")
    fine = torch.ones(40, 4, dtype=torch.bool)
    fine[7, 2] = fine[30, 1] = False
    for t in (y, d["dx"], d["dgate"]):
        assert torch.isfinite(t.cpu()[fine]).all() and torch.isnan(t.cpu()[7, 2]).any()


def test_two_runs_give_the_same_bits(gdp):
    x, w, b, z, dy = (dev(t) for t in make(5001, 16, 128, BF16, weight="channel", bias=True, seed=9))
    runs = [gdp.group_norm_backward(x, dy, w, b, z, "silu") for _ in range(3)]
    for r in runs[1:]:
        assert all(torch.equal(r[k], runs[0][k]) for k in r)


def test_many_tokens(gdp):
    """The weight gradients of many rows, against float64 sums on the GPU."""
    T, G, V = 20011, 8, 128
    x, w, b, z, dy = (dev(t) for t in make(T, G, V, BF16, weight="head", bias=True, seed=10))
    d = gdp.group_norm_backward(x, dy, w, b, z, "silu", False)
    xf, zf, df = x.double(), z.double(), dy.double()
    xhat = xf * ((xf * xf).mean(-1, keepdim=True) + 1e-5) ** -0.5
    dn = df * zf * torch.sigmoid(zf)
    for name, term in (("dweight", dn * xhat), ("dbias", dn)):
        # each term is good to 100 U (its factors' bounds), a sum of R terms to (R / 64 + 64) U
        limit = (term.abs().sum((0, 1)) * (T * G / 64 + 164) * layers.U).cpu()
        assert ((d[name].double() - term.sum((0, 1))).abs().cpu() <= limit).all(), name


def test_offsets_past_32_bits(gdp):
    T, G, V = 600000, 32, 128
    x = torch.ones(T, G, V, dtype=BF16, device="cuda")
    tail = torch.randn(4, G, V).to(BF16)
    x[-4:] = tail.cuda()
    y = gdp.group_norm(x, activation="silu", subtract_mean=False)
    want = layers.norm(tail, activation="silu", subtract_mean=False, d_y=tail)
    close(y[-4:], want["y"], want["y_bound"], "y", BF16)
    d = gdp.group_norm_backward(x, x, activation="silu", subtract_mean=False)
    close(d["dx"][-4:], want["dx"], want["dx_bound"], "dx", BF16)


def test_gradients_against_differences(gdp):
    """Central differences of the kernel's own forward pass; the truncation error from two exact ones."""
    x, w, b, z, dy = make(6, 2, 48, F32, bias=True, seed=11)
    gen = torch.Generator().manual_seed(12)
    d = gdp.group_norm_backward(x.cuda(), dy.cuda(), w.cuda(), b.cuda(), z.cuda(), "silu")
    noise = float((layers.norm(x, w, b, z, "silu")["y_bound"] * dy.abs()).sum())
    s = 2.0 ** -6
    for at, name in enumerate(("dx", "dweight", "dbias", "dgate")):
        args = [x, w, b, z]
        v = torch.randn(args[at].shape, generator=gen)

        def loss(step, exact):
            moved = list(args)
            moved[at] = args[at] + step * v
            if exact:
                y = layers.norm(*moved, "silu")["y"]
            else:
                y = gdp.group_norm(*(t.cuda() for t in moved), "silu").cpu().double()
            return float((y * dy.double()).sum())

        got = (loss(s, False) - loss(-s, False)) / (2 * s)
        one = (loss(s, True) - loss(-s, True)) / (2 * s)
        two = (loss(2 * s, True) - loss(-2 * s, True)) / (4 * s)
        want = float((d[name].cpu().double() * v).sum())
        assert abs(got - want) <= abs(two - one) + 2 * noise / s, (name, got, want, abs(two - one), noise / s)


def test_graph_replay_and_streams(gdp):
    x, w, b, z, dy = (dev(t) for t in make(600, 6, 100, BF16, weight="channel", bias=True, seed=13))
    T, G, V = x.shape
    y, dx, dz = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    dw, db = torch.empty(G, V, device="cuda"), torch.empty(G, V, device="cuda")
    ws = torch.empty(gdp.gdp_group_norm_backward_workspace_bytes(T, G, V), dtype=torch.uint8, device="cuda")

    def body():
        gdp.gdp_group_norm(x, w, b, z, "silu", True, 1e-5, y)
        gdp.gdp_group_norm_backward(x, w, b, z, "silu", True, 1e-5, dy, dx, dw, db, dz, ws)

    body()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()
    for seed in range(3):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)))
        for t in (y, dx, dz, dw, db):
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, dx, dz, dw, db)]
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            for t in (y, dx, dz, dw, db):
                t.fill_(7.0)
            body()
        torch.cuda.synchronize()
        for p, q in zip(got, (y, dx, dz, dw, db)):
            assert torch.equal(p, q)


# ------------------------------------------------------------ layers together

def test_scan_then_norm_and_back(gdp):
    """A vector-state layer, forward and backward: recurrence, output norm with a swish gate; the norm's dx is
    the recurrence's d_o.  The reference takes each stage's stored result as the next one's input."""
    H, V = 4, 64
    lens, D = [90, 1, 0, 150], H * V
    gen = torch.Generator().manual_seed(14)
    T, cu = sum(lens), torch.tensor([0, 90, 91, 91, 241], dtype=torch.int32)
    x, z, dy = (torch.randn(T, D, generator=gen).to(BF16) for _ in range(3))
    g = -torch.nn.functional.softplus(torch.randn(T, D, generator=gen) - 3)
    w = 1 + 0.2 * torch.randn(V, generator=gen)
    o, fs, cp = gdp.gated_scan(x.cuda(), g.cuda(), cu.cuda(), output_final_state=True, complement_input=True,
                               return_checkpoints=True)
    heads = lambda t: t.view(T, H, V)  # noqa: E731
    form = dict(weight=w.cuda(), gate=heads(z).cuda(), activation="silu", subtract_mean=False)
    y = gdp.group_norm(heads(o), **form)
    d = gdp.group_norm_backward(heads(o), heads(dy).cuda(), **form)
    ds = gdp.gated_scan_backward(x.cuda(), g.cuda(), cu.cuda(), d["dx"].view(T, D), complement_input=True,
                                 checkpoints=cp)
    ref = layers.scan(x, g, cu.tolist(), None, True)
    close(o, ref["o"], ref["o_bound"], "o", BF16)
    want = layers.norm(heads(o.cpu()), w, None, heads(z), "silu", False, d_y=heads(dy))
    close(y, want["y"], want["y_bound"], "y", BF16)
    close(d["dx"], want["dx"], want["dx_bound"], "dx", BF16)
    close(d["dgate"], want["dgate"], want["dgate_bound"], "dgate", BF16)
    close(d["dweight"], want["dweight"], want["dweight_bound"], "dweight", F32)
    back = layers.scan_backward(x, g, cu.tolist(), d["dx"].view(T, D).cpu(), None, None, True)
    close(ds["dx"], back["dx"], back["dx_bound"], "scan dx", F32)
    close(ds["dg_log"], back["dg"], back["dg_bound"], "scan dg", F32)


def test_prefill_then_norm_and_back(gdp):
    """The norm on the matrix-state prefill's outputs, its dx as d_o of the prefill's gradients, and a decode
    step's output through the same norm."""
    from gated_deltaproduct_recurrence_amd import workloads
    wl = workloads.custom([70, 33], 2, 1, 2, 64, 64, init_std=0.2, seed=15)
    inp = {k: dev(v) if isinstance(v, torch.Tensor) else v for k, v in workloads.generate(wl, "cpu").items()}
    o, fs = gdp.chunk_prefill(**inp)
    T, H, V = o.shape
    gen = torch.Generator().manual_seed(16)
    z, dy = (torch.randn(T, H, V, generator=gen).to(BF16) for _ in range(2))
    w = 1 + 0.2 * torch.randn(V, generator=gen)
    form = dict(weight=w.cuda(), gate=z.cuda(), activation="silu", subtract_mean=False)
    y = gdp.group_norm(o, **form)
    want = layers.norm(o.cpu(), w, None, z, "silu", False, d_y=dy)
    close(y, want["y"], want["y_bound"], "y", BF16)
    d = gdp.group_norm_backward(o, dy.cuda(), **form)
    close(d["dx"], want["dx"], want["dx_bound"], "dx", BF16)
    grads = gdp.chunk_prefill_backward(inp["q"], inp["k"], inp["v"], inp["g_log"], inp["beta"], 2, inp["cu_seqlens"],
                                       d["dx"], initial_state=inp["initial_state"])
    assert all(torch.isfinite(t).all() for t in grads.values() if t is not None)
    cache = fs.clone()
    slots = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    od = gdp.recurrent_decode(inp["q"][:2], inp["k"][:4], inp["v"][:4], inp["g_log"][:2], inp["beta"][:4], 2, cache, slots)
    yd = gdp.group_norm(od, w.cuda(), gate=z[:2].cuda(), activation="silu", subtract_mean=False)
    wd = layers.norm(od.cpu(), w, None, z[:2], "silu", False)
    close(yd, wd["y"], wd["y_bound"], "y", BF16)


def test_captured_layer_step(gdp):
    """The allocating front ends of a whole layer step (scan, norm, both gradients) captured into a graph; each
    replay, with new inputs and eager work in between, gives the eager step's bits."""
    H, V = 3, 64
    lens, D = [190, 0, 70], H * V
    T = sum(lens)
    cu = torch.tensor([0, 190, 190, 260], dtype=torch.int32, device="cuda")
    gen = torch.Generator().manual_seed(18)
    x, z, dy = (torch.randn(T, D, generator=gen).to(BF16).cuda() for _ in range(3))
    g = -torch.rand(T, D, generator=gen).cuda()
    w = (1 + 0.2 * torch.randn(V, generator=gen)).cuda()

    def step():
        heads = lambda t: t.view(T, H, V)  # noqa: E731
        o, fs, cp = gdp.gated_scan(x, g, cu, output_final_state=True, return_checkpoints=True)
        form = dict(weight=w, gate=heads(z), activation="silu", subtract_mean=False)
        y = gdp.group_norm(heads(o), **form)
        d = gdp.group_norm_backward(heads(o), heads(dy), **form)
        ds = gdp.gated_scan_backward(x, g, cu, d["dx"].view(T, D), checkpoints=cp, grads_like_inputs=True)
        return [y, fs, d["dgate"], d["dweight"], ds["dx"], ds["dg_log"]]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(4):
        x.copy_(torch.randn(T, D, generator=gen))
        dy.copy_(torch.randn(T, D, generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
