"""The operators around a recurrence run as a layer uses them: projections, short convolution, recurrence, norms between
blocks; prompt, next token and training step (needs a gfx950 GPU)."""
import pytest
import torch

from oracle import blocks
from tests.test_gpu_short_conv import close, edges

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def gdp():
    from gated_deltaproduct_recurrence_amd import binding
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return binding


def layer(D=64, M=96, S=8, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    return dict(D=D, M=M, S=S, w_in=rand(M, 2 * D) / M ** 0.5, w_x=rand(D, D + 2 * S) / D ** 0.5, w_out=rand(D, M) / D ** 0.5,
                conv_w=rand(D, 4) * 0.5, conv_b=rand(D) * 0.1, A=-(rand(D, S).abs() + 0.1), skip=rand(D), bias=rand(D) - 2,
                post=1 + 0.1 * rand(M), pre=1 + 0.1 * rand(M))


def forward(gdp, p, x, n, cu, s_conv=None, s_scan=None):
    """Residual stream x and normed input n [T, M] through one layer of this kind: what the next layer gets."""
    D, S = p["D"], p["S"]
    xz = n @ p["w_in"]
    u, conv_state = gdp.short_conv(xz[:, :D], p["conv_w"], cu, bias=p["conv_b"], activation="silu", initial_state=s_conv,
                                   output_final_state=True)
    proj = u @ p["w_x"]
    B, C = proj[:, D:D + S].unsqueeze(1), proj[:, D + S:].unsqueeze(1)
    o, scan_state = gdp.selective_scan(u, proj[:, :D], p["A"], B, C, cu, skip=p["skip"], gate=xz[:, D:], dt_bias=p["bias"],
                                       dt_softplus=True, initial_state=s_scan, output_final_state=True)
    r, n = gdp.residual_norm(x, o @ p["w_out"], p["post"], p["pre"], residual_scale=0.5)
    return r, n, conv_state, scan_state


def test_a_prompt_in_pieces_and_token_by_token(gdp):
    """Strided projections as inputs; a prompt in two calls with carried states, then single tokens on the caches, against
    the whole in one call.  float32 throughout: the ways differ by their sums' order alone."""
    p = layer()
    gen = torch.Generator().manual_seed(1)
    lens, cut = [40, 3, 29], [17, 3, 8]
    cu = edges(lens)
    x, n = torch.randn(cu[-1], p["M"], generator=gen).cuda(), torch.randn(cu[-1], p["M"], generator=gen).cuda()
    whole = forward(gdp, p, x, n, torch.tensor(cu, device="cuda"))
    first = torch.cat([torch.arange(cu[i], cu[i] + cut[i]) for i in range(3)]).cuda()
    rest = torch.cat([torch.arange(cu[i] + cut[i], cu[i + 1]) for i in range(3)]).cuda()
    a = forward(gdp, p, x[first], n[first], torch.tensor(edges(cut), device="cuda"))
    left = [m - c for m, c in zip(lens, cut)]
    b = forward(gdp, p, x[rest], n[rest], torch.tensor(edges(left), device="cuda"), a[2], a[3])
    for i in (0, 1):
        both = torch.empty_like(whole[i])
        both[first], both[rest] = a[i], b[i]
        assert torch.allclose(both, whole[i], rtol=1e-4, atol=1e-4)
    assert torch.allclose(b[2], whole[2], rtol=1e-5, atol=1e-5) and torch.allclose(b[3], whole[3], rtol=1e-4, atol=1e-4)
    # one more token per sequence on caches, entry 1 padding
    D, S = p["D"], p["S"]
    conv_cache, scan_cache = whole[2].clone(), whole[3].clone()
    slots = torch.tensor([0, -1, 2], device="cuda")
    xt, nt = torch.randn(3, p["M"], generator=gen).cuda(), torch.randn(3, p["M"], generator=gen).cuda()
    xz = nt @ p["w_in"]
    u = gdp.short_conv_decode(xz[:, :D], p["conv_w"], conv_cache, slots, bias=p["conv_b"], activation="silu")
    proj = u @ p["w_x"]
    o = gdp.selective_scan_decode(u, proj[:, :D], p["A"], proj[:, D:D + S].unsqueeze(1), proj[:, D + S:].unsqueeze(1),
                                  scan_cache, slots, skip=p["skip"], gate=xz[:, D:], dt_bias=p["bias"], dt_softplus=True)
    r, nn = gdp.residual_norm(xt, o @ p["w_out"], p["post"], p["pre"], residual_scale=0.5, out=xt.clone())
    step = forward(gdp, p, xt, nt, torch.tensor([0, 1, 2, 3], device="cuda"), whole[2], whole[3])
    for i in (0, 2):
        assert torch.allclose(r[i], step[0][i], rtol=1e-4, atol=1e-4) and torch.allclose(nn[i], step[1][i], rtol=1e-4, atol=1e-4)
        assert torch.allclose(scan_cache[i], step[3][i], rtol=1e-4, atol=1e-4) and torch.equal(conv_cache[i], step[2][i])
    assert torch.equal(conv_cache[1], whole[2][1]) and torch.equal(scan_cache[1], whole[3][1])


def test_training_step(gdp):
    """The gradients of the chain, operator by operator in reverse, against autograd in float64 on the same formulas."""
    p = layer(D=32, M=48, S=4, seed=2)
    D, S, M = p["D"], p["S"], p["M"]
    gen = torch.Generator().manual_seed(3)
    lens = [19, 1, 44]
    cu = edges(lens)
    T = cu[-1]
    x, n, dr, dn = (torch.randn(T, M, generator=gen).cuda() for _ in range(4))
    cud = torch.tensor(cu, device="cuda")
    xz = n @ p["w_in"]
    conv = dict(bias=p["conv_b"], activation="silu")
    u, _ = gdp.short_conv(xz[:, :D], p["conv_w"], cud, **conv)
    proj = u @ p["w_x"]
    dt, B, C = proj[:, :D], proj[:, D:D + S].unsqueeze(1), proj[:, D + S:].unsqueeze(1)
    scan = dict(skip=p["skip"], gate=xz[:, D:], dt_bias=p["bias"], dt_softplus=True)
    o, _, points = gdp.selective_scan(u, dt, p["A"], B, C, cud, return_checkpoints=True, **scan)
    y = o @ p["w_out"]
    norms = dict(post_weight=p["post"], pre_weight=p["pre"], residual_scale=0.5)
    g3 = gdp.residual_norm_backward(x, y, dr, dn, **norms)
    g2 = gdp.selective_scan_backward(u, dt, p["A"], B, C, cud, g3["dy"] @ p["w_out"].t(), checkpoints=points, **scan)
    dproj = torch.cat([g2["ddt"], g2["dB"][:, 0], g2["dC"][:, 0]], 1)
    g1 = gdp.short_conv_backward(xz[:, :D], p["conv_w"], cud, g2["du"] + dproj @ p["w_x"].t(), **conv)
    got = dict(n=torch.cat([g1["dx"], g2["dgate"]], 1) @ p["w_in"].t(), x=g3["dx"], conv_w=g1["dweight"], conv_b=g1["dbias"],
               A=g2["dA"], skip=g2["dskip"], bias=g2["ddt_bias"], post=g3["dpost_weight"], pre=g3["dpre_weight"],
               w_out=o.t() @ g3["dy"], w_x=u.t() @ dproj)

    q = {k: v.detach().cpu().double().requires_grad_() for k, v in {**{k: v for k, v in p.items() if torch.is_tensor(v)},
                                                                   "x": x, "n": n}.items()}
    XZ = q["n"] @ q["w_in"]
    pieces = []
    for lo, hi in zip(cu, cu[1:]):
        rows = torch.cat([torch.zeros(3, D, dtype=torch.float64), XZ[lo:hi, :D]])
        pieces.append(sum(rows[j:j + hi - lo] * q["conv_w"][:, j] for j in range(4)) + q["conv_b"])
    U = torch.nn.functional.silu(torch.cat(pieces))
    P = U @ q["w_x"]
    delta = torch.nn.functional.softplus(P[:, :D] + q["bias"])
    O = []
    for lo, hi in zip(cu, cu[1:]):
        h = torch.zeros(D, S, dtype=torch.float64)
        for t in range(lo, hi):
            h = torch.exp(delta[t][:, None] * q["A"]) * h + (delta[t] * U[t])[:, None] * P[t, D:D + S]
            O.append((h * P[t, D + S:]).sum(1) + q["skip"] * U[t])
    Y = (torch.stack(O) * torch.nn.functional.silu(XZ[:, D:])) @ q["w_out"]
    norm = lambda v, w: v * (v.pow(2).mean(-1, keepdim=True) + 1e-5).rsqrt() * w  # noqa: E731
    R = q["x"] + 0.5 * norm(Y, q["post"])
    loss = (R * dr.cpu()).sum() + (norm(R, q["pre"]) * dn.cpu()).sum()
    loss.backward()
    for k, t in got.items():
        want = q[k].grad
        assert (t.cpu().double() - want).norm() <= 1e-5 * want.norm(), k


def test_before_the_matrix_state_recurrence(gdp):
    """The convolution's outputs as queries, keys and values of the prefill: the same as of a convolution formed apart."""
    gen = torch.Generator().manual_seed(5)
    lens, H, K = [37, 64, 130], 2, 64
    cu = edges(lens)
    T, D = cu[-1], 3 * H * K
    x, w = torch.randn(T, D, generator=gen).to(BF16), torch.randn(D, 4, generator=gen) * 0.5
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, _ = gdp.short_conv(x.cuda(), w.cuda(), cud, activation="silu")
    want = blocks.conv(x, w, cu, None, "silu")
    close(y, want["y"], want["y_bound"], "y", BF16)
    q, k, v = (t.reshape(T, H, K) for t in y.split(H * K, 1))
    g, beta = -torch.rand(T, H, generator=gen).cuda(), torch.rand(T, H, generator=gen).cuda()
    o, fs = gdp.chunk_prefill(q, k, v, g, beta, 1, cud, output_final_state=True, use_qk_l2norm=True)
    o2, fs2 = gdp.chunk_prefill(*(t.contiguous() for t in (q, k, v)), g, beta, 1, cud, output_final_state=True,
                                use_qk_l2norm=True)
    assert torch.equal(o, o2) and torch.equal(fs, fs2) and torch.isfinite(o.float()).all()


def test_two_captured_calls_share_a_workspace_in_order(gdp):
    """Two graphs captured on one workspace and one stream, replayed in turn, each leave the eager results."""
    gen = torch.Generator().manual_seed(6)
    T, D, S = 300, 72, 8
    ins = []
    for _ in range(2):
        t = [torch.randn(T, D, generator=gen).cuda(), torch.randn(T, D, generator=gen).cuda(), -torch.rand(D, S, generator=gen).cuda() - 0.1,
             torch.randn(T, 1, S, generator=gen).cuda(), torch.randn(T, 1, S, generator=gen).cuda()]
        ins.append(t)
    cu = torch.tensor([0, 200, 300], dtype=torch.int32, device="cuda")
    ws = torch.empty(gdp.gdp_selective_scan_workspace_bytes(T, 2, D, 1, S), dtype=torch.uint8, device="cuda")
    outs = [torch.empty(T, D, device="cuda") for _ in range(2)]

    def call(i):
        gdp.gdp_selective_scan(*ins[i], None, None, None, True, cu, None, False, None, None, False, outs[i], None, None, ws)

    eager = [gdp.selective_scan(*t, cu, dt_softplus=True)[0] for t in ins]
    graphs = []
    for i in range(2):
        call(i)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i)
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, e) for o, e in zip(outs, eager))


def test_debug_validation_covers_these_entries(gdp, monkeypatch):
    monkeypatch.setenv("GDP_DEBUG_VALIDATE", "1")
    gdp.gdp_debug_status()
    x, w = torch.randn(10, 8, device="cuda"), torch.randn(8, 4, device="cuda")
    gdp.short_conv(x, w, torch.tensor([0, 4, 10], device="cuda"))
    assert gdp.gdp_debug_status() == 0
    gdp.short_conv(x, w, torch.tensor([0, 11], device="cuda"))
    assert gdp.gdp_debug_status() == gdp.GDP_DBG_CU
    cache = torch.zeros(4, 8, 2, device="cuda")
    A, B = -torch.ones(8, 2, device="cuda"), torch.randn(10, 1, 2, device="cuda")
    gdp.selective_scan(x, x, A, B, B, torch.tensor([0, 4, 10], device="cuda"), state_cache=cache,
                       state_indices=torch.tensor([1, 9], device="cuda"))
    assert gdp.gdp_debug_status() == gdp.GDP_DBG_SLOT
    gdp.short_conv_decode(x[:2], w, torch.zeros(4, 3, 8, device="cuda"), torch.tensor([-1, -2], device="cuda"))
    assert gdp.gdp_debug_status() == gdp.GDP_DBG_SLOT


def test_boundaries_that_do_not_rise_stay_in_bounds(gdp):
    """Bad boundaries give wrong rows and nothing else: results for the sequences' own shapes, neighbours untouched."""
    T, D, S = 90, 24, 4
    x, w = torch.randn(T, D, device="cuda"), torch.randn(D, 4, device="cuda")
    A, B = -torch.ones(D, S, device="cuda"), torch.randn(T, 1, S, device="cuda")
    for bad in ([0, 50, 20, 90], [90, 0, 90, 40], [-5, 30, 200, 60]):
        cu = torch.tensor(bad, device="cuda")
        guard = torch.full((T + 200, D), 2.0, device="cuda")
        y, fs = gdp.short_conv(x, w, cu, output_final_state=True, out=guard[100:100 + T])
        o, fs, points = gdp.selective_scan(x, x, A, B, B, cu, dt_softplus=True, output_final_state=True,
                                           return_checkpoints=True, out=guard[100:100 + T])
        gdp.selective_scan_backward(x, x, A, B, B, cu, x, dt_softplus=True, checkpoints=points)
        gdp.short_conv_backward(x, w, cu, x)
        assert (guard[:100] == 2).all() and (guard[100 + T:] == 2).all()
