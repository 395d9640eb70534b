"""The norms around a block with gate, residual scale and residual sum, and their gradients, through the binding against
the float64 oracle (needs a gfx950 GPU)."""
import pytest
import torch

from oracle import blocks
from tests.test_gpu_short_conv import close, dev

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def gdp():
    from gated_deltaproduct_recurrence_amd import binding
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return binding


def make(T, D, dtype, stream=None, gated=True, wdtype=F32, post_w=True, pre_w=True, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    st = stream or dtype
    return dict(x=rand(T, D).to(st), y=(0.5 * rand(T, D) + 0.1).to(dtype), z=rand(T, D).to(dtype) if gated else None,
                wa=(1 + 0.3 * rand(D)).to(wdtype) if post_w else None, wb=(1 + 0.3 * rand(D)).to(wdtype) if pre_w else None,
                dr=rand(T, D).to(st), dn=rand(T, D).to(dtype))


def check(gdp, d, act=None, post=True, pre=True, scale=0.5, eps=1e-5, with_dr=True, on=None):
    on = on or {k: dev(v) for k, v in d.items()}
    form = dict(activation=act, post_norm=post, pre_norm=pre, residual_scale=scale, eps=eps)
    dr, dn = (d["dr"] if with_dr else None), (d["dn"] if pre else None)
    want = blocks.residual_norm(d["x"], d["y"], d["wa"], d["wb"], d["z"], d_r=dr, d_n=dn, **form)
    weights = dict(post_weight=on["wa"], pre_weight=on["wb"], gate=on["z"])
    r, n = gdp.residual_norm(on["x"], on["y"], **weights, **form)
    close(r, want["r"], want["r_bound"], "r", d["x"].dtype)
    if pre:
        close(n, want["n"], want["n_bound"], "n", d["y"].dtype)
    else:
        assert n is None
    g = gdp.residual_norm_backward(on["x"], on["y"], on["dr"] if with_dr else None, on["dn"] if pre else None, **weights,
                                   **form)
    close(g["dx"], want["dx"], want["dx_bound"], "dx", d["x"].dtype)
    close(g["dy"], want["dy"], want["dy_bound"], "dy", d["y"].dtype)
    for name, given, dtype in (("dgate", d["z"], d["y"].dtype), ("dpost_weight", d["wa"], F32), ("dpre_weight", d["wb"], F32)):
        if given is None:
            assert g[name] is None
        else:
            close(g[name], want[name], want[name + "_bound"], name, dtype)
    return r, n, g


@pytest.mark.parametrize("D", [1, 2, 3, 7, 8, 9, 31, 63, 64, 96, 255, 256, 257, 511, 512, 513, 1000, 1024, 1025, 2000, 2049])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_channel_counts(gdp, D, dtype):
    check(gdp, make(9, D, dtype, seed=D), "sigmoid")


@pytest.mark.parametrize("D", [4096, 5001, 8192, 8200, 16384])
@pytest.mark.parametrize("dtype,stream", [(F32, F32), (BF16, F32)])
def test_wide(gdp, D, dtype, stream):
    check(gdp, make(5, D, dtype, stream, seed=D), "silu")


@pytest.mark.parametrize("dtype,stream", [(F32, F32), (BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)])
@pytest.mark.parametrize("D", [128, 90, 1500])
@pytest.mark.parametrize("own", [False, True])
def test_types(gdp, dtype, stream, D, own):
    check(gdp, make(37, D, dtype, stream, wdtype=dtype if own else F32, seed=1), "silu")


@pytest.mark.parametrize("act", [None, "none", "silu", "sigmoid"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_forms(gdp, act, post, pre, weights, gated):
    d = make(21, 200, F32, gated=gated, post_w=weights, pre_w=weights and pre, seed=2)
    act = act if gated else None
    check(gdp, d, act, post, pre, scale=-0.75)
    check(gdp, d, act, post, pre, scale=1.0, with_dr=not pre)


@pytest.mark.parametrize("T", [0, 1, 3, 300, 4099, 20000])
def test_token_counts(gdp, T):
    check(gdp, make(T, 64, F32, seed=3), "sigmoid")
    if T < 1000:
        check(gdp, make(T, 2100, BF16, seed=4), "sigmoid")


def test_strides(gdp):
    """Operands as slices of wider buffers that start anywhere, a gate shared by the tokens, outputs in wider buffers."""
    d = make(50, 77, BF16, F32, seed=5)
    on = {k: dev(v) for k, v in d.items()}
    for k, at in (("x", 1), ("y", 3), ("dr", 5), ("dn", 7)):
        wide = torch.zeros(50, 100, dtype=d[k].dtype, device="cuda")
        wide[:, at:at + 77] = on[k]
        on[k] = wide[:, at:at + 77]
    d["z"] = d["z"][:1].expand(50, 77)
    on["z"] = on["z"][:1].expand(50, 77)
    check(gdp, d, "sigmoid", on=on)
    want = blocks.residual_norm(d["x"], d["y"], d["wa"], d["wb"], residual_scale=2.0)
    r, n = torch.full((50, 90), 3.0, device="cuda"), torch.full((50, 81), 3.0, dtype=BF16, device="cuda")
    gdp.gdp_residual_norm(on["x"], on["y"], on["wa"], on["wb"], None, None, True, True, 2.0, 1e-5, r[:, 13:], n[:, 1:78])
    close(r[:, 13:], want["r"], want["r_bound"], "r", F32)
    close(n[:, 1:78], want["n"], want["n_bound"], "n", BF16)
    assert (r[:, :13] == 3).all() and (n[:, 0] == 3).all() and (n[:, 78:] == 3).all()


@pytest.mark.parametrize("D", [64, 1001, 4096])
def test_in_place(gdp, D):
    d = make(33, D, BF16, seed=6)
    form = dict(post_weight=dev(d["wa"]), pre_weight=dev(d["wb"]), gate=dev(d["z"]), activation="sigmoid")
    r, n = gdp.residual_norm(dev(d["x"]), dev(d["y"]), **form)
    wide = torch.zeros(33, D + 5, dtype=BF16, device="cuda")
    x = wide[:, 2:2 + D]
    x.copy_(d["x"])
    r2, n2 = gdp.residual_norm(x, dev(d["y"]), out=x, **form)
    assert torch.equal(x, r) and torch.equal(n2, n) and r2.data_ptr() == x.data_ptr()
    assert (wide[:, :2] == 0).all() and (wide[:, 2 + D:] == 0).all()


def test_rows_of_zeros_and_far_gates(gdp):
    """Tokens whose y, or whose residual stream, is all zeros: the norm of nothing is nothing, and its gradient finite."""
    d = make(16, 300, F32, seed=7)
    d["y"][3], d["x"][5], d["y"][5], d["z"] = 0.0, 0.0, 0.0, d["z"] * 60.0
    for act in ("silu", "sigmoid"):
        r, n, g = check(gdp, d, act)
        assert (n[5] == 0).all() and torch.isfinite(g["dy"]).all()


def test_a_bad_value_stays_in_its_token(gdp):
    d = make(40, 128, F32, seed=8)
    d["y"][7, 5], d["x"][30, 0] = float("nan"), float("inf")
    on = {k: dev(v) for k, v in d.items()}
    form = dict(post_weight=on["wa"], pre_weight=on["wb"], gate=on["z"], activation="silu")
    r, n = gdp.residual_norm(on["x"], on["y"], **form)
    g = gdp.residual_norm_backward(on["x"], on["y"], on["dr"], on["dn"], **form)
    fine = torch.ones(40, dtype=torch.bool)
    fine[7] = fine[30] = False
    for t in (r, n, g["dx"], g["dy"], g["dgate"]):
        assert torch.isfinite(t.cpu()[fine]).all()
    assert torch.isnan(n.cpu()[7]).any() and torch.isnan(n.cpu()[30]).any()


def test_streams_graphs_and_repeats(gdp):
    d = make(700, 2560, BF16, F32, seed=9)
    on = {k: dev(v) for k, v in d.items()}
    form = dict(post_weight=on["wa"], pre_weight=on["wb"], gate=on["z"], activation="sigmoid")

    def both():
        r, n = gdp.residual_norm(on["x"], on["y"], **form)
        return [r, n, *gdp.residual_norm_backward(on["x"], on["y"], on["dr"], on["dn"], **form).values()]

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
    for seed in (10, 11, 12):
        new = make(700, 2560, BF16, F32, seed=seed)
        for k in ("x", "y", "dr", "dn", "z"):
            on[k].copy_(new[k])
        eager = both()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(held, eager))
