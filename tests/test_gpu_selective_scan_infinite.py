"""Infinite inputs of the selective scan: a prompt and its tokens one by one give what the formula gives, also where there
is no skip and where the states do not fill what a kernel holds (needs a gfx950 GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")
LENS = [3, 16, 45]
EDGES = [0, 3, 19, 64]


@pytest.fixture(scope="module")
def gdp():
    from gated_deltaproduct_recurrence_amd import binding
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return binding


def make(S, dtype, skip, D=70):
    """Positive inputs, so that sums of infinities are infinite; decays that keep a state for hundreds of rows."""
    gen = torch.Generator().manual_seed(S)
    rand = lambda *s: torch.rand(*s, generator=gen) + 0.5  # noqa: E731
    d = dict(u=rand(64, D), dt=0.1 * rand(64, D), A=-0.3 * rand(D, S), B=rand(64, 1, S), C=rand(64, 1, S),
             skip=rand(D) if skip else None, z=torch.randn(64, D, generator=gen))
    d["u"][1, 2] = d["u"][18, 3] = d["u"][40, 4] = d["u"][21, 5] = d["u"][19, 6] = INF
    d["u"][63, 7] = -INF
    d["dt"][50, 8] = d["dt"][25, 9] = INF
    return {k: v if v is None or k in ("A", "skip") else v.to(dtype) for k, v in d.items()}


def formula(d):
    u, dt, A, B, C, z = (d[k].double() for k in ("u", "dt", "A", "B", "C", "z"))
    o, final = [], []
    for lo, hi in zip(EDGES, EDGES[1:]):
        h = torch.zeros_like(A)
        for t in range(lo, hi):
            h = torch.exp(dt[t][:, None] * A) * h + (dt[t] * u[t])[:, None] * B[t]
            y = (h * C[t]).sum(1)
            if d["skip"] is not None:
                y = y + d["skip"].double() * u[t]
            o.append(y * z[t] * torch.sigmoid(z[t]))
        final.append(h)
    return torch.stack(o), torch.stack(final)


def alike(got, want, what):
    """The same infinities and numbers in the same places (the numbers themselves are compared elsewhere)."""
    got = got.detach().cpu().double()
    for name, f in (("+inf", lambda t: t == INF), ("-inf", lambda t: t == -INF), ("nan", torch.isnan)):
        bad = f(got) != f(want)
        assert not bad.any(), (what, name, torch.nonzero(bad)[:3].tolist(), got[bad][:3], want[bad][:3])


@pytest.mark.parametrize("S", [1, 2, 3, 4, 5, 8, 9, 12, 16, 17, 24, 31, 32])
@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompt_and_steps(gdp, S, skip, dtype):
    d = make(S, dtype, skip)
    on = {k: None if v is None else v.cuda() for k, v in d.items()}
    o, final = formula(d)
    assert (o == INF).any() and (o == -INF).any()
    cu = torch.tensor(EDGES, device="cuda")
    got, fs = gdp.selective_scan(on["u"], on["dt"], on["A"], on["B"], on["C"], cu, skip=on["skip"], gate=on["z"],
                                 output_final_state=True)
    alike(got, o, "prompt")
    alike(fs, final, "final state")
    cache = torch.zeros(3, *d["A"].shape, device="cuda")
    for t in range(max(LENS)):
        live = [i for i in range(3) if LENS[i] > t]
        rows = torch.tensor([EDGES[i] + t for i in live], device="cuda")
        step = gdp.selective_scan_decode(on["u"][rows], on["dt"][rows], on["A"], on["B"][rows], on["C"][rows], cache,
                                         torch.tensor(live, device="cuda"), skip=on["skip"], gate=on["z"][rows])
        alike(step, o[rows.cpu()], "step")
        alike(step, got[rows].cpu().double(), "step and prompt")
    alike(cache, final, "cache")


@pytest.mark.parametrize("S", [4, 16])
def test_the_gates_gradient_without_a_skip(gdp, S):
    """d gate = d_o silu'(gate) (C . h): infinite with the state."""
    d = make(S, F32, False)
    d["dt"] = d["dt"].nan_to_num(posinf=0.1)
    on = {k: None if v is None else v.cuda() for k, v in d.items()}
    cu = torch.tensor(EDGES, device="cuda")
    g = gdp.selective_scan_backward(on["u"], on["dt"], on["A"], on["B"], on["C"], cu, torch.ones_like(on["u"]), gate=on["z"])
    z = d["z"].double()
    s = torch.sigmoid(z)
    slope = s + z * s * (1 - s)
    for t, ch in ((1, 2), (18, 3), (40, 4), (21, 5), (19, 6)):
        assert g["dgate"][t, ch] == (INF if slope[t, ch] > 0 else -INF)
