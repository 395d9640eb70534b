"""Dimensions of one element with strides of their own, as torch's contiguous() leaves them: the results are those of
plain tensors (needs a gfx950 GPU)."""
import pytest
import torch

from tests.test_gpu_gated_scan import BF16, F32, gdp, make  # noqa: F401

pytestmark = pytest.mark.gpu


def odd(t):
    """t [.., 1] with another stride in its last dimension."""
    wide = torch.zeros(*t.shape[:-1], 5, dtype=t.dtype, device="cuda")
    wide[..., 2:3] = t.cuda()
    view = torch.as_strided(wide, t.shape, (*wide.stride()[:-1], 3), 2)
    assert view.stride(-1) == 3 and torch.equal(view.cpu(), t.cpu())
    return view


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_a_slot_out_of_a_table(gdp, index):  # noqa: F811
    table = torch.full((4, 7), -1, dtype=index, device="cuda")
    table[0, 3] = 2
    slot = table[:1, 3].contiguous()
    assert slot.stride() == (7,)
    x, g, cu, s0 = make([130], 96, BF16, F32, seed=1)
    x, g, cu, s0 = (t.cuda() for t in (x, g, cu, s0))
    start = torch.randn(5, 96, device="cuda")
    got, want = [], []
    for out, s in ((got, slot), (want, slot + 0)):
        cache = start.clone()
        o, _ = gdp.gated_scan(x, g, cu, initial_state=s0, state_cache=cache, state_indices=s)
        out += [o, gdp.gated_scan_decode(x[:1], g[:1], cache, s), cache]
        H, K = 2, 64
        gen = torch.Generator(device="cuda").manual_seed(3)
        q, k, v = (torch.randn(1, H, K, generator=gen, device="cuda").to(BF16) for _ in range(3))
        gl, beta = -torch.rand(1, H, generator=gen, device="cuda"), torch.rand(1, H, generator=gen, device="cuda")
        states = torch.randn(5, H, K, K, generator=gen, device="cuda")
        out += [gdp.recurrent_decode(q, k, v, gl, beta, 1, states, s), states]
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_one_channel(gdp):  # noqa: F811
    x, g, cu, s0 = make([200, 57, 1], 1, F32, F32, seed=2)
    a = gdp.gated_scan(x.cuda(), g.cuda(), cu.cuda(), initial_state=s0.cuda(), output_final_state=True)
    b = gdp.gated_scan(odd(x), odd(g), cu.cuda(), initial_state=s0.cuda(),
                       output_final_state=True)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    da = gdp.gated_scan_backward(x.cuda(), g.cuda(), cu.cuda(), x.cuda(), initial_state=s0.cuda())
    db = gdp.gated_scan_backward(odd(x), odd(g), cu.cuda(), odd(x), initial_state=s0.cuda())
    assert all(torch.equal(da[n], db[n]) for n in da)


def test_groups_of_one(gdp):  # noqa: F811
    x, z = torch.randn(50, 6, 1), torch.randn(50, 6, 1)
    w, b = torch.randn(6, 1), torch.randn(6, 1)
    form = dict(activation="silu", subtract_mean=False)
    plain = dict(weight=w.cuda(), bias=b.cuda(), gate=z.cuda(), **form)
    other = dict(weight=torch.as_strided(w.cuda(), (6, 1), (1, 9)), bias=b.cuda(), gate=odd(z), **form)
    assert torch.equal(gdp.group_norm(x.cuda(), **plain), gdp.group_norm(odd(x), **other))
    da, db = gdp.group_norm_backward(x.cuda(), x.cuda(), **plain), gdp.group_norm_backward(odd(x), odd(x), **other)
    assert all(torch.equal(da[n], db[n]) for n in da)


def test_one_state_head(gdp):  # noqa: F811
    """Gates [T, 1] of the matrix-state recurrence, prefill and gradients (those of the gates are summed by LDS atomics
    in any order, so their bits are not compared)."""
    T, K = 150, 64
    gen = torch.Generator().manual_seed(4)
    q, k, v = (torch.nn.functional.normalize(torch.randn(T, 1, K, generator=gen), dim=-1).to(BF16).cuda() for _ in range(3))
    gl, beta = -torch.rand(T, 1, generator=gen), torch.rand(T, 1, generator=gen)
    cu = torch.tensor([0, 100, T], dtype=torch.int32, device="cuda")
    runs = []
    for f in (lambda t: t.cuda(), odd):
        o, fs = gdp.chunk_prefill(q, k, v, f(gl), f(beta), 1, cu, output_final_state=True)
        d = gdp.chunk_prefill_backward(q, k, v, f(gl), f(beta), 1, cu, q)
        runs.append([o, fs, d["dq"], d["dk"], d["dv"]])
    for a, b in zip(*runs):
        assert torch.equal(a, b)
