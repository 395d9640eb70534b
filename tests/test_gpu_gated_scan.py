"""The gated linear recurrence (scan, single-token step, gradients) through the binding against the float64
oracle (needs a gfx950 GPU).  Tolerances are the oracle's element-wise bounds plus the stored type's rounding."""
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


def make(lens, D, dtype, gate, seed=0, initial=True, first=0, behind=0, shift=3.0):
    """Inputs on the CPU; `first` rows before the first sequence, `behind` behind the last."""
    gen = torch.Generator().manual_seed(seed)
    T, N = first + sum(lens) + behind, len(lens)
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    x = torch.randn(T, D, generator=gen).to(dtype)
    g = (-torch.nn.functional.softplus(torch.randn(T, D, generator=gen) - shift)).to(gate)
    s0 = torch.randn(N, D, generator=gen) if initial else None
    return x, g, torch.tensor(cu, dtype=torch.int32), s0


def dev(t):
    return None if t is None else t.cuda()


def close(got, value, bound, what):
    got = got.detach().cpu().to(torch.float64)
    limit = layers.rounded(value, bound, what[1])
    bad = ~((got - value).abs() <= limit)
    assert not bad.any(), (what[0], int(bad.sum()), tuple(torch.nonzero(bad)[0].tolist()),
                           float(got[bad][0]), float(value[bad][0]), float(limit[bad][0]))


def check_scan(gdp, x, g, cu, s0, complement, xd=None, gd=None, out=None):
    """Forward and backward of one set of inputs; xd, gd: other device layouts of x and g."""
    T, D = x.shape
    N = cu.numel() - 1
    ref = layers.scan(x, g, cu.tolist(), s0, complement)
    xd, gd, cud = dev(x) if xd is None else xd, dev(g) if gd is None else gd, dev(cu)
    lo, hi = (int(cu[0]), int(cu[-1]))
    o = torch.full((T, D), 77.0, dtype=x.dtype, device="cuda") if out is None else out
    o, fs, points = gdp.gated_scan(xd, gd, cud, initial_state=dev(s0), output_final_state=True,
                                   complement_input=complement, return_checkpoints=True, out=o)
    torch.cuda.synchronize()
    close(o[lo:hi], ref["o"][lo:hi], ref["o_bound"][lo:hi], ("o", x.dtype))
    close(fs, ref["final"], ref["final_bound"], ("final", F32))
    assert (o[:lo] == 77).all() and (o[hi:] == 77).all(), "rows outside the sequences were written"
    starts = set(cu.tolist())
    for c in range(points.shape[0]):
        t = 64 * c
        if lo <= t < hi and t not in starts:
            close(points[c], ref["before"][t], ref["before_bound"][t], ("checkpoint %d" % c, F32))
    gen = torch.Generator().manual_seed(99)
    d_o = torch.randn(T, D, generator=gen).to(x.dtype)
    d_final = torch.randn(N, D, generator=gen) if s0 is not None else None
    want = layers.scan_backward(x, g, cu.tolist(), d_o, d_final, s0, complement)
    for cp, like in ((points, False), (None, True)):
        r = gdp.gated_scan_backward(xd, gd, cud, dev(d_o), d_final_state=dev(d_final), initial_state=dev(s0),
                                    complement_input=complement, checkpoints=cp, grads_like_inputs=like)
        torch.cuda.synchronize()
        close(r["dx"], want["dx"], want["dx_bound"], ("dx", x.dtype if like else F32))
        close(r["dg_log"], want["dg"], want["dg_bound"], ("dg", g.dtype if like else F32))
        if s0 is not None:
            close(r["d_initial_state"], want["ds0"], want["ds0_bound"], ("ds0", F32))
        else:
            assert r["d_initial_state"] is None


LENGTHS = [[1], [63], [64], [65], [127], [128], [129], [128, 256, 1], [1] * 200, [0, 5, 0, 0, 130, 0], [200, 57, 64, 128, 1], [700], []]


@pytest.mark.parametrize("lens", LENGTHS, ids=lambda v: "x".join(map(str, v[:6])) or "none")
@pytest.mark.parametrize("complement", [False, True])
def test_lengths(gdp, lens, complement):
    check_scan(gdp, *make(lens, 40, BF16, F32, seed=len(lens)), complement)


@pytest.mark.parametrize("D", [1, 3, 64, 100, 255, 256, 260, 1001])
def test_channel_counts(gdp, D):
    check_scan(gdp, *make([70, 3, 150], D, BF16, F32, seed=D), False)


@pytest.mark.parametrize("dtype,gate", [(F32, F32), (BF16, F32), (BF16, BF16), (F16, F32), (F16, F16)])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("D", [48, 515])
def test_types(gdp, dtype, gate, complement, D):
    check_scan(gdp, *make([130, 1, 0, 77], D, dtype, gate, seed=5), complement)


@pytest.mark.parametrize("initial", [False, True])
def test_rows_outside_the_sequences(gdp, initial):
    x, g, cu, s0 = make([100, 30], 72, BF16, F32, initial=initial, first=75, behind=133)
    x[:75], x[-133:], g[:75], g[-133:] = float("nan"), float("inf"), float("nan"), float("nan")
    check_scan(gdp, x, g, cu, s0, True)


@pytest.mark.parametrize("count", [511, 512, 513, 3000])
def test_many_short_sequences(gdp, count):
    lens = [(7 * i * i + i) % 4 for i in range(count)]
    check_scan(gdp, *make(lens, 8, F32, F32, seed=count), False)


def test_many_empty_sequences(gdp):
    check_scan(gdp, *make([0] * 1500 + [70] + [0] * 1500 + [1, 65], 12, F32, F32), False)


def test_very_many_sequences(gdp):
    """More than 512 x 512 sequences, mostly empty: the search for a tile's sequences takes two steps."""
    N, D = 300000, 4
    lens = torch.zeros(N, dtype=torch.int64)
    lens[500::1000] = 3
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)])
    gen = torch.Generator().manual_seed(24)
    T = int(cu[-1])
    x, g, s0 = torch.randn(T, D, generator=gen), -torch.rand(T, D, generator=gen), torch.randn(N, D, generator=gen)
    full = lens > 0
    ref = layers.scan(x, g, list(range(0, T + 1, 3)), s0[full])
    o, fs = gdp.gated_scan(x.cuda(), g.cuda(), cu.cuda(), initial_state=s0.cuda(), output_final_state=True)
    close(o, ref["o"], ref["o_bound"], ("o", F32))
    close(fs[full.cuda()], ref["final"], ref["final_bound"], ("final", F32))
    assert torch.equal(fs[~full.cuda()].cpu(), s0[~full])
    d = gdp.gated_scan_backward(x.cuda(), g.cuda(), cu.cuda(), x.cuda(), d_final_state=s0.cuda(), initial_state=s0.cuda())
    want = layers.scan_backward(x, g, list(range(0, T + 1, 3)), x, s0[full], s0[full])
    close(d["dx"], want["dx"], want["dx_bound"], ("dx", F32))
    close(d["d_initial_state"][full.cuda()], want["ds0"], want["ds0_bound"], ("ds0", F32))
    assert torch.equal(d["d_initial_state"][~full.cuda()].cpu(), s0[~full])


@pytest.mark.parametrize("D", [96, 131])
def test_strided_gradients_and_decode_rows(gdp, D):
    """Gradients and single-token rows inside wider buffers, through the direct calls."""
    x, g, cu, s0 = make([90, 64, 33], D, BF16, BF16, seed=25, first=5, behind=9)
    T, N = x.shape[0], 3
    d_o = torch.randn(T, D, generator=torch.Generator().manual_seed(26)).to(BF16)
    want = layers.scan_backward(x, g, cu.tolist(), d_o, None, s0)
    wide = {k: torch.full((T, D + 7), 9.0, dtype=t, device="cuda") for k, t in (("do", BF16), ("dx", F32), ("dg", BF16))}
    wide["do"][:, 3:3 + D] = d_o.cuda()
    views = {k: t[:, 3:3 + D] for k, t in wide.items()}
    ds0 = torch.empty(N, D, device="cuda")
    ws = torch.empty(gdp.gdp_gated_scan_backward_workspace_bytes(T, N, D), dtype=torch.uint8, device="cuda")
    gdp.gdp_gated_scan_backward(x.cuda(), g.cuda(), cu.cuda(), False, s0.cuda(), None, views["do"], None, views["dx"],
                                views["dg"], ds0, ws)
    close(views["dx"], want["dx"], want["dx_bound"], ("dx", F32))
    close(views["dg"], want["dg"], want["dg_bound"], ("dg", BF16))
    close(ds0, want["ds0"], want["ds0_bound"], ("ds0", F32))
    for k in ("dx", "dg"):
        assert (wide[k][:, :3] == 9).all() and (wide[k][:, 3 + D:] == 9).all(), k
    cache, slots = torch.randn(8, D), torch.tensor([7, 1, 4])
    ref = layers.decode(x[:3], g[:3], cache, slots, True)
    xw, ow = (torch.full((3, D + 5), 9.0, dtype=BF16, device="cuda") for _ in range(2))
    xw[:, 2:2 + D] = x[:3].cuda()
    cd = cache.cuda()
    gdp.gated_scan_decode(xw[:, 2:2 + D], g[:3].cuda(), cd, slots.cuda(), complement_input=True, out=ow[:, 2:2 + D])
    close(ow[:, 2:2 + D], ref["o"], ref["o_bound"], ("o", BF16))
    close(cd, ref["cache"], ref["cache_bound"], ("cache", F32))
    assert (ow[:, :2] == 9).all() and (ow[:, 2 + D:] == 9).all()


def test_operands_elsewhere_are_refused(gdp):
    x, g = torch.randn(10, 8, device="cuda"), -torch.rand(10, 8, device="cuda")
    with pytest.raises(ValueError, match="expected a tensor on cuda"):
        gdp.gated_scan(x, g, torch.tensor([0, 10], dtype=torch.int32))
    with pytest.raises(ValueError, match="expected a tensor on cuda"):
        gdp.gated_scan_decode(x, g, torch.zeros(10, 8, device="cuda"), torch.zeros(10, dtype=torch.int32))
    with pytest.raises(ValueError, match="expected a workspace on cuda"):
        gdp.gdp_gated_scan(x, g, torch.tensor([0, 10], dtype=torch.int32, device="cuda"), False, None, False, None, None,
                           False, torch.empty_like(x), None, None, torch.empty(4096, dtype=torch.uint8))
    with pytest.raises(ValueError, match="unsupported dtype"):
        gdp.gated_scan(x.double(), g, torch.tensor([0, 10], dtype=torch.int32, device="cuda"))
    with pytest.raises(gdp.GdpError, match="x and o must share one dtype"):
        gdp.gated_scan(x, g, torch.tensor([0, 10], dtype=torch.int32, device="cuda"), out=torch.empty_like(x, dtype=BF16))


def test_int64_boundaries_and_strided_rows(gdp):
    x, g, cu, s0 = make([90, 64, 33], 96, BF16, F32, seed=8)
    T, D = x.shape
    wide = torch.randn(T, 3 * D, device="cuda").to(BF16)
    wide[:, D:2 * D] = x.cuda()
    gw = torch.randn(T, D + 4, device="cuda")
    gw[:, :D] = g.cuda()
    ow = torch.full((T, D + 8), 77.0, dtype=BF16, device="cuda")
    check_scan(gdp, x, g, cu.long(), s0, False, xd=wide[:, D:2 * D], gd=gw[:, :D], out=ow[:, 8:])
    assert (ow[:, :8] == 77).all()


def test_rows_that_no_vector_width_aligns(gdp):
    x, g, cu, s0 = make([90, 64, 33], 96, BF16, F32, seed=9)
    T, D = x.shape
    flat = torch.empty(T * (D + 1) + 1, dtype=BF16, device="cuda")
    xd = flat[1:].view(T, D + 1)[:, :D]
    xd.copy_(x)
    check_scan(gdp, x, g, cu, s0, True, xd=xd)


def test_gates_broadcast_over_the_tokens(gdp):
    """One row of decays for all tokens (row stride 0); the gradient has a row for each token."""
    x, g, cu, s0 = make([90, 64, 33], 96, F32, F32, seed=10)
    g = g[:1].expand(x.shape[0], -1)
    check_scan(gdp, x, g, cu, s0, False, gd=g[:1].cuda().expand(x.shape[0], -1))


def test_extreme_gates(gdp):
    """-inf restarts a channel; 0 keeps a running sum; strong decays underflow."""
    x, g, cu, s0 = make([300, 140], 64, F32, F32, seed=11)
    g[:, :16] = 0.0
    g[::7, 16:32] = float("-inf")
    g[:, 32:48] *= 400.0
    check_scan(gdp, x, g, cu, s0, False)
    check_scan(gdp, x, g, cu, s0, True)


def test_a_bad_value_stays_in_its_sequence_and_channel(gdp):
    x, g, cu, s0 = make([100, 200, 150], 64, F32, F32, seed=12)
    x[120, 5], x[250, 6], s0[1, 7] = float("nan"), float("inf"), float("nan")
    o, fs = gdp.gated_scan(x.cuda(), g.cuda(), cu.cuda(), initial_state=s0.cuda(), output_final_state=True)
    good_x, good_s = torch.nan_to_num(x, 0, 0), torch.nan_to_num(s0, 0)
    ref = layers.scan(good_x, g, cu.tolist(), good_s)
    fine = torch.ones_like(x, dtype=torch.bool)
    fine[100:300, 5:8] = False
    assert torch.isfinite(o.cpu()[fine]).all()
    limit = layers.rounded(ref["o"], ref["o_bound"], F32)
    assert ((o.cpu().double() - ref["o"]).abs() <= limit)[fine].all()
    assert torch.isnan(o[120:300, 5]).all() and torch.isinf(o[250:300, 6]).all() and torch.isnan(o[100:300, 7]).all()
    ok = torch.ones_like(s0, dtype=torch.bool)
    ok[1, 5:8] = False
    assert torch.isfinite(fs.cpu()[ok]).all()


@pytest.mark.parametrize("D", [40, 600])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 100.0])
def test_a_bad_gate_stays_in_its_sequence_and_channel(gdp, D, bad):
    """A decay that is not finite, in a tile that holds the end of one sequence and a part of the next:
    neither the next one's states nor the gradients of the one before see it, to the bit."""
    x, g, cu, s0 = make([150, 450], D, F32, F32, seed=21)
    d_o, d_final = torch.randn_like(x), torch.randn_like(s0)
    worse = g.clone()
    worse[130, 3] = bad  # the first sequence's, in the tile's first wave
    worse[190, 5] = bad  # the second one's, in the last wave of a tile of 64 rows
    got = []
    for gates in (g, worse):
        o, fs, points = gdp.gated_scan(x.cuda(), gates.cuda(), cu.cuda(), initial_state=s0.cuda(),
                                       output_final_state=True, return_checkpoints=True)
        r = gdp.gated_scan_backward(x.cuda(), gates.cuda(), cu.cuda(), d_o.cuda(), d_final_state=d_final.cuda(),
                                    initial_state=s0.cuda(), checkpoints=points)
        got.append({"o": o.cpu(), "fs": fs.cpu(), **{k: v.cpu() for k, v in r.items()}})
    good, poor = got
    rows = torch.ones_like(x, dtype=torch.bool)
    rows[:150, 3] = False
    rows[150:, 5] = False
    states = torch.ones_like(s0, dtype=torch.bool)
    states[0, 3] = states[1, 5] = False
    for name, value in good.items():
        where = states if name in ("fs", "d_initial_state") else rows
        assert torch.equal(poor[name][where], value[where]), name


def test_no_rows(gdp):
    x, g = torch.empty(0, 24, device="cuda"), torch.empty(0, 24, device="cuda")
    s0 = torch.randn(3, 24, device="cuda")
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    o, fs, points = gdp.gated_scan(x, g, cu, initial_state=s0, output_final_state=True, return_checkpoints=True)
    assert o.shape == (0, 24) and points.shape == (0, 24) and torch.equal(fs, s0)
    d = gdp.gated_scan_backward(x, g, cu, o, d_final_state=s0, initial_state=s0, checkpoints=points)
    assert torch.equal(d["d_initial_state"], s0)


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_state_cache(gdp, index):
    x, g, cu, s0 = make([90, 0, 1, 200, 30], 130, BF16, F32, seed=13)
    slots = torch.tensor([6, 2, -1, 0, 9], dtype=index)  # 9 is past the cache of 8
    cache = torch.randn(8, 130)
    cd = cache.cuda()
    _, fs = gdp.gated_scan(x.cuda(), g.cuda(), cu.cuda(), initial_state=s0.cuda(), output_final_state=True,
                           state_cache=cd, state_indices=slots.cuda())
    for i, s in ((0, 6), (1, 2), (3, 0)):
        assert torch.equal(cd[s], fs[i])
    left = [1, 3, 4, 5, 7]
    assert torch.equal(cd[left].cpu(), cache[left])
    cd2 = cache.cuda()
    gdp.gated_scan(x.cuda(), g.cuda(), cu.cuda(), initial_state=s0.cuda(), state_cache=cd2,
                   state_indices=slots.cuda())
    assert torch.equal(cd, cd2)


def test_a_continued_sequence_is_the_whole_one(gdp):
    """A sequence cut in two, the second part from the first part's final state."""
    x, g, cu, _ = make([500], 256, BF16, F32, seed=14, initial=False)
    o, fs = gdp.gated_scan(x.cuda(), g.cuda(), cu.cuda(), output_final_state=True)
    ref = layers.scan(x, g, [0, 500])
    one = lambda n: torch.tensor([0, n], dtype=torch.int32, device="cuda")  # noqa: E731
    o1, f1 = gdp.gated_scan(x[:211].cuda(), g[:211].cuda(), one(211), output_final_state=True)
    o2, f2 = gdp.gated_scan(x[211:].cuda(), g[211:].cuda(), one(289), initial_state=f1, output_final_state=True)
    close(torch.cat([o1, o2]), ref["o"], ref["o_bound"], ("o", BF16))
    close(f2, ref["final"], ref["final_bound"], ("final", F32))
    close(o, ref["o"], ref["o_bound"], ("o", BF16))


@pytest.mark.parametrize("lens,first,behind", [([9000, 300, 11000], 0, 0), ([2048, 4096, 100, 1948, 1024], 0, 300),
                                               ([5000, 0, 1, 3000], 2100, 0)])
def test_long_axis_few_channels(gdp, lens, first, behind):
    """Hundreds of blocks handed on through groups in one channel block; sequences that end with a group."""
    x, g, cu, s0 = make(lens, 5, F32, F32, seed=15, shift=6.0, first=first, behind=behind)
    check_scan(gdp, x, g, cu, s0, False)


@pytest.mark.parametrize("D,dtype,gate,complement", [(700, F32, F32, True), (769, BF16, F32, False), (640, F16, F16, True)])
def test_long_axis_many_channels(gdp, D, dtype, gate, complement):
    """Many blocks handed on in more than four channel blocks; the last of 769 channels is alone in its block."""
    x, g, cu, s0 = make([2500, 1, 700, 129], D, dtype, gate, seed=23, shift=5.0)
    check_scan(gdp, x, g, cu, s0, complement)


def test_two_runs_give_the_same_bits(gdp):
    x, g, cu, s0 = (dev(t) for t in make([5000, 1, 3000, 900], 512, BF16, F32, seed=16))
    d_o = torch.randn(x.shape, device="cuda").to(BF16)
    runs = []
    for _ in range(3):
        o, fs, cp = gdp.gated_scan(x, g, cu, initial_state=s0, output_final_state=True, return_checkpoints=True)
        d = gdp.gated_scan_backward(x, g, cu, d_o, initial_state=s0, checkpoints=cp)
        runs.append([o, fs, d["dx"], d["dg_log"], d["d_initial_state"]])
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def test_offsets_past_32_bits(gdp):
    """More than 2^32 bytes and 2^31 elements in x: the last rows against the oracle."""
    T, D = 70016, 32768
    lens = [T - 100, 100]
    x = torch.zeros(T, D, dtype=BF16, device="cuda")
    x[::1000] = 1.0
    g = torch.full((1, D), -0.05, device="cuda").expand(T, D)
    tail = torch.randn(100, D, device="cuda").to(BF16)
    x[-100:] = tail
    cu = torch.tensor([0, T - 100, T], dtype=torch.int32, device="cuda")
    o, fs, cp = gdp.gated_scan(x, g, cu, output_final_state=True, return_checkpoints=True)
    cols = torch.tensor([0, 1, 255, 256, 16383, 32767])
    ref = layers.scan(tail[:, cols.cuda()], g[:100, cols.cuda()], [0, 100])
    close(o[-100:, cols.cuda()], ref["o"], ref["o_bound"], ("o", BF16))
    before = layers.scan(x[-1500:-100][:, cols.cuda()], g[:1400, cols.cuda()], [0, 1400])  # exp(-0.05 1400) < 2^-100
    close(fs[0, cols.cuda()][None], before["final"], before["final_bound"], ("final", F32))
    d_o = torch.zeros_like(x)
    d_o[-100:] = tail
    d = gdp.gated_scan_backward(x, g, cu, d_o, checkpoints=cp, grads_like_inputs=True)
    want = layers.scan_backward(tail[:, cols.cuda()], g[:100, cols.cuda()], [0, 100], tail[:, cols.cuda()])
    close(d["dx"][-100:, cols.cuda()], want["dx"], want["dx_bound"], ("dx", BF16))
    close(d["dg_log"][-100:, cols.cuda()], want["dg"], want["dg_bound"], ("dg", F32))
    assert not d["dx"][:T - 100].any()


def test_gradients_against_differences(gdp):
    """The outputs are linear in x and in the initial state: differences over a step of 1 are exact but for
    rounding.  In g the loss has third derivatives below (its effective memory)^3 |h e|; a central
    difference over a step s is off by s^2 / 6 of that."""
    x, g, cu, s0 = make([100, 64, 37], 32, F32, F32, seed=17, shift=1.0)
    gen = torch.Generator().manual_seed(18)
    d_o, d_f = torch.randn(x.shape, generator=gen), torch.randn(s0.shape, generator=gen)
    d = gdp.gated_scan_backward(x.cuda(), g.cuda(), cu.cuda(), d_o.cuda(), d_final_state=d_f.cuda(),
                                initial_state=s0.cuda())

    def loss(x, g, s0):
        o, fs = gdp.gated_scan(x.cuda(), g.cuda(), cu.cuda(), initial_state=s0.cuda(), output_final_state=True)
        return ((o.cpu().double() * d_o.double()).sum(), (fs.cpu().double() * d_f.double()).sum())

    base = layers.scan(x, g, cu.tolist(), s0)
    noise = float((base["o_bound"] * d_o.abs()).sum() + (base["final_bound"] * d_f.abs()).sum())
    vx, vs = torch.randn(x.shape, generator=gen), torch.randn(s0.shape, generator=gen)
    up, down = loss(x + vx, g, s0 + vs), loss(x - vx, g, s0 - vs)
    got = (sum(up) - sum(down)) / 2
    want = (d["dx"].cpu().double() * vx).sum() + (d["d_initial_state"].cpu().double() * vs).sum()
    # each side's evaluation is off by at most `noise` scaled by the larger inputs (|x| + |v| <= 8)
    assert abs(got - want) <= 8 * noise, (float(got), float(want), noise)
    vg = torch.randn(g.shape, generator=gen)
    s = 2.0 ** -6
    up, down = loss(x, g + s * vg, s0), loss(x, g - s * vg, s0)
    got = (sum(up) - sum(down)) / (2 * s)
    want = (d["dg_log"].cpu().double() * vg).sum()
    exact = []
    for k in (1, 2):  # the truncation error from two exact central differences: their difference is 3/4 of the larger's
        vals = []
        for sign in (1, -1):
            f = layers.scan(x, g + sign * k * s * vg, cu.tolist(), s0)
            vals.append(float((f["o"] * d_o.double()).sum() + (f["final"] * d_f.double()).sum()))
        exact.append((vals[0] - vals[1]) / (2 * k * s))
    truncation = abs(exact[1] - exact[0])
    assert abs(got - want) <= truncation + 2 * noise / s, (float(got), float(want), truncation, noise / s)


def test_other_streams_and_workspaces(gdp):
    """Two calls at once on two streams."""
    sets = [[dev(t) for t in make([3000, 500, 900], 1024, BF16, F32, seed=s)] for s in (19, 20)]
    plain = [gdp.gated_scan(x, g, cu, initial_state=s0, output_final_state=True) for x, g, cu, s0 in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(3):
        for st, (x, g, cu, s0) in zip(streams, sets):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(gdp.gated_scan(x, g, cu, initial_state=s0, output_final_state=True))
    torch.cuda.synchronize()
    for k, (o, fs) in enumerate(got):
        assert torch.equal(o, plain[k % 2][0]) and torch.equal(fs, plain[k % 2][1])


def test_graph_replay(gdp):
    """Forward pass, gradients and single-token step captured with shared workspaces in two graphs; each replay,
    with new boundaries and eager work between them, gives the eager result."""
    x, g, cu, s0 = (dev(t) for t in make([700, 300, 24], 256, BF16, F32, seed=21))
    d_o = torch.randn(x.shape, device="cuda").to(BF16)
    T, D = x.shape
    N = 3
    ws = torch.empty(gdp.gdp_gated_scan_backward_workspace_bytes(T, N, D), dtype=torch.uint8, device="cuda")
    o, fs = torch.empty_like(x), torch.empty(N, D, device="cuda")
    dx, dg, ds0 = (torch.empty(*s, device="cuda") for s in ((T, D), (T, D), (N, D)))
    cache, slots = torch.zeros(4, D, device="cuda"), torch.tensor([3, 0, 1], dtype=torch.int32, device="cuda")
    od = torch.empty(N, D, dtype=BF16, device="cuda")

    def forward():
        gdp.gdp_gated_scan(x, g, cu, False, s0, True, cache, slots, False, o, fs, None, ws)
        gdp.gdp_gated_scan_decode(x[:N], g[:N], False, cache, slots, od)

    def backward():
        gdp.gdp_gated_scan_backward(x, g, cu, False, s0, None, d_o, None, dx, dg, ds0, ws)

    forward()
    backward()
    torch.cuda.synchronize()
    graphs = []
    for body in (forward, backward):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            body()
        graphs.append(graph)
    for cuts in ([0, 700, 1000, 1024], [0, 1, 513, 1024], [10, 74, 74, 1000], [0, 0, 0, 1024]):
        cu.copy_(torch.tensor(cuts, dtype=torch.int32))
        for t in (o, fs, dx, dg, ds0, od):
            t.fill_(7.0)
        cache.zero_()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (o, fs, dx, dg, ds0, od, cache)]
        for t in (o, fs, dx, dg, ds0, od):
            t.fill_(7.0)
        cache.zero_()
        forward()
        backward()
        torch.cuda.synchronize()
        for a, b in zip(got, (o, fs, dx, dg, ds0, od, cache)):
            assert torch.equal(a, b), cuts


def test_bad_boundaries_stay_in_bounds(gdp):
    """Decreasing boundaries and entries outside [0, T] give wrong numbers, nothing else: guard rows around
    every buffer keep their values."""
    T, D, N = 200, 64, 4

    def guarded(rows, dtype, cols=D):
        big = torch.full((rows + 16, cols), 5.0, dtype=dtype, device="cuda")
        return big, big[8:8 + rows]

    x, g = torch.randn(T, D, device="cuda"), -torch.rand(T, D, device="cuda")
    for cuts in ([0, 150, 100, 180, 200], [-50, 10, 999, 40, 5000], [200, 150, 100, 50, 0], [300, 300, 300, 300, 300]):
        cu = torch.tensor(cuts, dtype=torch.int32, device="cuda")
        bufs = {k: guarded(r, F32) for k, r in (("o", T), ("fs", N), ("cp", 4), ("dx", T), ("dg", T), ("ds0", N),
                                                ("cache", 3))}
        ws = torch.empty(gdp.gdp_gated_scan_backward_workspace_bytes(T, N, D), dtype=torch.uint8, device="cuda")
        slots = torch.tensor([0, -5, 7, 2], dtype=torch.int64, device="cuda")
        b = {k: v[1] for k, v in bufs.items()}
        gdp.gdp_gated_scan(x, g, cu, False, None, True, b["cache"], slots, True, b["o"], b["fs"], b["cp"], ws)
        gdp.gdp_gated_scan_backward(x, g, cu, True, None, b["cp"], x, None, b["dx"], b["dg"], b["ds0"], ws)
        gdp.gdp_gated_scan_backward(x, g, cu, True, None, None, x, None, b["dx"], b["dg"], b["ds0"], ws)
        torch.cuda.synchronize()
        for k, (big, inner) in bufs.items():
            assert (big[:8] == 5).all() and (big[8 + inner.shape[0]:] == 5).all(), (cuts, k)


DECODE = [(1, 1, F32, F32), (1, 256, BF16, F32), (5, 100, BF16, BF16), (64, 1001, F16, F16), (33, 513, F16, F32)]


@pytest.mark.parametrize("N,D,dtype,gate", DECODE)
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_decode(gdp, N, D, dtype, gate, complement, index):
    gen = torch.Generator().manual_seed(N)
    x = torch.randn(N, D, generator=gen).to(dtype)
    g = (-torch.nn.functional.softplus(torch.randn(N, D, generator=gen) - 3)).to(gate)
    cache = torch.randn(N + 3, D, generator=gen)
    slots = torch.randperm(N + 3, generator=gen)[:N].to(index)
    if N > 3:
        slots[1], slots[3] = -1, N + 3
    ref = layers.decode(x, g, cache, slots, complement)
    cd = cache.cuda()
    o = gdp.gated_scan_decode(x.cuda(), g.cuda(), cd, slots.cuda(), complement_input=complement)
    close(o, ref["o"], ref["o_bound"], ("o", dtype))
    close(cd, ref["cache"], ref["cache_bound"], ("cache", F32))
    named = [int(s) for s in slots if 0 <= s < N + 3]
    left = [s for s in range(N + 3) if s not in named]
    assert torch.equal(cd[left].cpu(), cache[left])


def test_decode_steps_equal_the_scan(gdp):
    T, D = 70, 260
    x, g, cu, s0 = make([T], D, BF16, F32, seed=22)
    ref = layers.scan(x, g, [0, T], s0)
    cache = torch.zeros(3, D, device="cuda")
    cache[2] = s0[0].cuda()
    slot = torch.tensor([2], dtype=torch.int32, device="cuda")
    o = torch.cat([gdp.gated_scan_decode(x[t:t + 1].cuda(), g[t:t + 1].cuda(), cache, slot) for t in range(T)])
    close(o, ref["o"], ref["o_bound"], ("o", BF16))
    close(cache[2:], ref["final"], ref["final_bound"], ("final", F32))


def test_debug_validation(gdp, monkeypatch):
    monkeypatch.setenv("GDP_DEBUG_VALIDATE", "1")
    gdp.gdp_debug_status()
    x, g = torch.randn(10, 8, device="cuda"), -torch.rand(10, 8, device="cuda")
    cu = torch.tensor([0, 6, 4], dtype=torch.int32, device="cuda")
    gdp.gated_scan(x, g, cu)
    assert gdp.gdp_debug_status() == gdp.GDP_DBG_CU
    cache = torch.zeros(4, 8, device="cuda")
    gdp.gated_scan_decode(x[:2], g[:2], cache, torch.tensor([4, 0], dtype=torch.int32, device="cuda"))
    assert gdp.gdp_debug_status() == gdp.GDP_DBG_SLOT
    gdp.gated_scan(x, g, torch.tensor([0, 6, 10], dtype=torch.int32, device="cuda"), state_cache=cache,
                   state_indices=torch.tensor([1, 2], dtype=torch.int32, device="cuda"))
    assert gdp.gdp_debug_status() == 0
