"""Refusals of the recurrence's and the norm's entry points: host-side checks, no GPU.  Pointers are fake,
never dereferenced: every call here fails validation before a launch."""
import ctypes

import pytest
import torch

from tests.test_abi_cpu import Fake


@pytest.fixture(scope="module")
def b():
    from gated_deltaproduct_recurrence_amd import binding
    return binding


def ref(t):
    return ctypes.byref(t) if t is not None else None


def scan_args(b, T=200, N=3, D=96, dt=None):
    f = Fake()
    dt = b.GDP_BF16 if dt is None else dt
    F32 = b.GDP_F32
    a = dict(x=f.tensor(b, dt, [T, D]), g=f.tensor(b, F32, [T, D]), cu=f.tensor(b, b.GDP_I32, [N + 1]), comp=0,
             s0=f.tensor(b, F32, [N, D]), ofs=1, cache=f.tensor(b, F32, [5, D]), slots=f.tensor(b, b.GDP_I32, [N]),
             rcp=1, o=f.tensor(b, dt, [T, D]), fs=f.tensor(b, F32, [N, D]), cp=f.tensor(b, F32, [-(-T // 64), D]),
             d_o=f.tensor(b, dt, [T, D]), df=f.tensor(b, F32, [N, D]), dx=f.tensor(b, F32, [T, D]),
             dg=f.tensor(b, F32, [T, D]), ds0=f.tensor(b, F32, [N, D]), ws=f.next, wsb=1 << 30)
    a["fake"] = f
    f.next += 1 << 31
    return a


def scan(b, a):
    return b.LIB.gdp_gated_scan(ref(a["x"]), ref(a["g"]), ref(a["cu"]), a["comp"], ref(a["s0"]), a["ofs"],
                                ref(a["cache"]), ref(a["slots"]), a["rcp"], ref(a["o"]), ref(a["fs"]), ref(a["cp"]),
                                a["ws"], a["wsb"], None)


def backward(b, a):
    return b.LIB.gdp_gated_scan_backward(ref(a["x"]), ref(a["g"]), ref(a["cu"]), a["comp"], ref(a["s0"]), ref(a["cp"]),
                                         ref(a["d_o"]), ref(a["df"]), ref(a["dx"]), ref(a["dg"]), ref(a["ds0"]),
                                         a["ws"], a["wsb"], None)


def decode(b, a):
    return b.LIB.gdp_gated_scan_decode(ref(a["x"]), ref(a["g"]), a["comp"], ref(a["cache"]), ref(a["slots"]),
                                       ref(a["o"]), None)


def refused(b, call, a, code, fragment):
    assert call(b, a) == code, b.gdp_last_error()
    assert fragment in b.gdp_last_error(), b.gdp_last_error()


def change(b, a, **new):
    """a with tensors replaced: name=(dtype, shape[, strides]), or None for absent."""
    for k, v in new.items():
        a[k] = None if v is None else a["fake"].tensor(b, *v)
    return a


BOTH = [scan, backward]


@pytest.mark.parametrize("call", BOTH)
def test_scan_missing_operands(b, call):
    for k, text in (("x", "required"), ("g", "required"), ("cu", "cu_seqlens is required")):
        refused(b, call, change(b, scan_args(b), **{k: None}), b.GDP_EINVAL, text)
    for k in ("o",) if call is scan else ("d_o", "dx", "dg"):
        refused(b, call, change(b, scan_args(b), **{k: None}), b.GDP_EINVAL, "required")


def test_scan_flags_need_their_buffers(b):
    refused(b, scan, change(b, scan_args(b), fs=None), b.GDP_EINVAL, "output_final_state needs")
    refused(b, scan, change(b, scan_args(b), cp=None), b.GDP_EINVAL, "return_checkpoints needs")
    refused(b, scan, change(b, scan_args(b), slots=None), b.GDP_EINVAL, "go together")
    refused(b, scan, change(b, scan_args(b), cache=None), b.GDP_EINVAL, "go together")


@pytest.mark.parametrize("call", BOTH)
def test_scan_shapes(b, call):
    refused(b, call, change(b, scan_args(b), x=(b.GDP_BF16, [200, 4, 24])), b.GDP_EINVAL, "x must be [T, D]")
    refused(b, call, change(b, scan_args(b), x=(b.GDP_BF16, [200, 0])), b.GDP_EINVAL, "at least one channel")
    refused(b, call, change(b, scan_args(b), g=(b.GDP_F32, [199, 96])), b.GDP_EINVAL, "g_log: dim 0")
    refused(b, call, change(b, scan_args(b), g=(b.GDP_F32, [200, 96], [192, 2])), b.GDP_EINVAL, "innermost")
    refused(b, call, change(b, scan_args(b), cu=(b.GDP_I32, [2, 2])), b.GDP_EINVAL, "cu_seqlens must be a contiguous")
    refused(b, call, change(b, scan_args(b), cu=(b.GDP_F32, [4])), b.GDP_EINVAL, "int32 or int64")
    refused(b, call, change(b, scan_args(b), s0=(b.GDP_F32, [4, 96])), b.GDP_EINVAL, "initial_state: dim 0")
    refused(b, call, change(b, scan_args(b), s0=(b.GDP_F32, [3, 96], [128, 1])), b.GDP_EINVAL, "contiguous")
    refused(b, call, change(b, scan_args(b), cp=(b.GDP_F32, [3, 96])), b.GDP_EINVAL, "checkpoints: dim 0")
    a = scan_args(b)
    a["x"].stride[0] = -96
    refused(b, call, a, b.GDP_EINVAL, "negative strides")


@pytest.mark.parametrize("call", BOTH)
def test_scan_types(b, call):
    refused(b, call, change(b, scan_args(b), x=(b.GDP_I32, [200, 96])), b.GDP_EUNSUPPORTED, "x must be")
    refused(b, call, change(b, scan_args(b), g=(b.GDP_F16, [200, 96])), b.GDP_EUNSUPPORTED, "g_log must be")
    refused(b, call, change(b, scan_args(b), s0=(b.GDP_BF16, [3, 96])), b.GDP_EUNSUPPORTED, "float32")
    if call is scan:
        refused(b, call, change(b, scan_args(b), o=(b.GDP_F32, [200, 96])), b.GDP_EUNSUPPORTED, "share one dtype")
    else:
        refused(b, call, change(b, scan_args(b), d_o=(b.GDP_F32, [200, 96])), b.GDP_EUNSUPPORTED, "share one dtype")
        refused(b, call, change(b, scan_args(b), dx=(b.GDP_F16, [200, 96])), b.GDP_EUNSUPPORTED, "dx must be")
        refused(b, call, change(b, scan_args(b), dg=(b.GDP_BF16, [200, 96])), b.GDP_EUNSUPPORTED, "dg_log must be")


def test_scan_overlaps(b):
    for out in ("o", "fs", "cp", "cache"):
        for other in ("x", "g", "s0", "cu", "slots"):
            a = scan_args(b)
            a[out].data = a[other].data
            refused(b, scan, a, b.GDP_EALIAS, "overlaps input")
    a = scan_args(b)
    a["fs"].data = a["cache"].data
    refused(b, scan, a, b.GDP_EALIAS, "overlaps")
    a = scan_args(b)
    a["ws"] = a["x"].data
    refused(b, backward, a, b.GDP_EALIAS, "workspace overlaps input x")
    a = change(b, scan_args(b), o=(b.GDP_BF16, [200, 96], [0, 1]))
    refused(b, scan, a, b.GDP_EALIAS, "its rows overlap")
    for out in ("dx", "dg", "ds0"):
        for other in ("x", "g", "d_o", "df", "cp"):
            a = scan_args(b)
            a[out].data = a[other].data
            refused(b, backward, a, b.GDP_EALIAS, "overlaps input")
    refused(b, backward, change(b, scan_args(b), dx=(b.GDP_F32, [200, 96], [95, 1])), b.GDP_EALIAS, "its rows overlap")


def test_scan_workspace(b):
    # more than 128 rows hand their states on through words: a counter and 8 bytes per tile and channel
    need = b.gdp_gated_scan_workspace_bytes(200, 3, 96)
    assert need >= 256 + 2 * 96 * 8
    a = scan_args(b)
    a["wsb"] = need - 1
    refused(b, scan, a, b.GDP_EWORKSPACE, "needed")
    a = scan_args(b)
    a["ws"] = a["o"].data
    refused(b, scan, a, b.GDP_EALIAS, "overlaps workspace")
    assert b.gdp_gated_scan_workspace_bytes(128, 3, 96) == 0
    # the gradients without checkpoints also form the states again
    need = b.gdp_gated_scan_backward_workspace_bytes(200, 3, 96)
    assert need >= 4 * 96 * 4
    a = scan_args(b)
    a["wsb"] = need - 1
    refused(b, backward, a, b.GDP_EWORKSPACE, "needed")
    a = scan_args(b)
    a["ws"] += 128
    refused(b, backward, a, b.GDP_EWORKSPACE, "aligned")
    a["ws"] = None
    refused(b, backward, a, b.GDP_EWORKSPACE, "needed")
    for bad in ((-1, 1, 8), (1, -1, 8), (1, 1, 0), (1 << 40, 1, 8), (1, 1, 1 << 24), (1 << 34, 1, 4096)):
        assert b.gdp_gated_scan_workspace_bytes(*bad) == 0
        assert b.gdp_gated_scan_backward_workspace_bytes(*bad) == 0


def test_scan_sizes_past_the_launch(b):
    """Sizes whose grid does not fit 32 bits are refused, with or without room for them."""
    a = change(b, scan_args(b, T=1 << 20, N=3, D=96), s0=None, cache=None, slots=None, fs=None, cp=None)
    a["ofs"], a["rcp"] = 0, 0
    for t in (a["x"], a["g"], a["o"]):
        t.shape[0], t.shape[1], t.stride[0] = 1 << 34, 4096, 0 if t is not a["o"] else 4096
    refused(b, scan, a, b.GDP_EUNSUPPORTED, "launch limits")


def test_launches_of_too_many_threads(b):
    """Each dimension of a launch holds less than 2^32 threads."""
    for bad in ((1 << 30, 1, 1), (1 << 26, 1, 1024), (1, 1 << 24, 8)):
        assert b.gdp_gated_scan_workspace_bytes(*bad) == 0
    assert b.gdp_gated_scan_workspace_bytes(1 << 28, 1, 1) > 0
    f = Fake()
    n = 1 << 24
    a = dict(x=f.tensor(b, b.GDP_BF16, [n, 1]), g=f.tensor(b, b.GDP_F32, [n, 1]), comp=0,
             cache=f.tensor(b, b.GDP_F32, [9, 1]), slots=f.tensor(b, b.GDP_I64, [n]),
             o=f.tensor(b, b.GDP_BF16, [n, 1]), fake=f)
    refused(b, decode, a, b.GDP_EUNSUPPORTED, "launch limits")


def test_decode_refusals(b):
    def args():
        f = Fake()
        return dict(x=f.tensor(b, b.GDP_BF16, [7, 96]), g=f.tensor(b, b.GDP_F32, [7, 96]), comp=0,
                    cache=f.tensor(b, b.GDP_F32, [9, 96]), slots=f.tensor(b, b.GDP_I64, [7]),
                    o=f.tensor(b, b.GDP_BF16, [7, 96]), fake=f)
    for k in ("x", "g", "o", "cache", "slots"):
        refused(b, decode, change(b, args(), **{k: None}), b.GDP_EINVAL, "required")
    refused(b, decode, change(b, args(), slots=(b.GDP_I64, [6])), b.GDP_EINVAL, "state_indices: dim 0")
    refused(b, decode, change(b, args(), slots=(b.GDP_F32, [7])), b.GDP_EINVAL, "int32 or int64")
    refused(b, decode, change(b, args(), cache=(b.GDP_F32, [9, 95])), b.GDP_EINVAL, "state_cache: dim 1")
    refused(b, decode, change(b, args(), cache=(b.GDP_BF16, [9, 96])), b.GDP_EUNSUPPORTED, "float32")
    refused(b, decode, change(b, args(), g=(b.GDP_F16, [7, 96])), b.GDP_EUNSUPPORTED, "g_log")
    a = args()
    a["o"].data = a["x"].data
    refused(b, decode, a, b.GDP_EALIAS, "o overlaps input x")
    a = args()
    a["o"].data = a["cache"].data
    refused(b, decode, a, b.GDP_EALIAS, "overlaps")


def norm_args(b, T=20, G=4, V=48, dt=None):
    f = Fake()
    dt = b.GDP_BF16 if dt is None else dt
    t3 = lambda: f.tensor(b, dt, [T, G, V])  # noqa: E731
    a = dict(x=t3(), w=f.tensor(b, b.GDP_F32, [V]), bias=f.tensor(b, b.GDP_F32, [V]), z=t3(), act=1, center=1, eps=1e-5,
             y=t3(), dy=t3(), dx=t3(), dw=f.tensor(b, b.GDP_F32, [V]), db=f.tensor(b, b.GDP_F32, [V]), dz=t3(),
             ws=f.next, wsb=1 << 30, fake=f)
    f.next += 1 << 31
    return a


def norm(b, a):
    return b.LIB.gdp_group_norm(ref(a["x"]), ref(a["w"]), ref(a["bias"]), ref(a["z"]), a["act"], a["center"], a["eps"],
                                ref(a["y"]), None)


def norm_backward(b, a):
    return b.LIB.gdp_group_norm_backward(ref(a["x"]), ref(a["w"]), ref(a["bias"]), ref(a["z"]), a["act"], a["center"],
                                         a["eps"], ref(a["dy"]), ref(a["dx"]), ref(a["dw"]), ref(a["db"]),
                                         ref(a["dz"]), a["ws"], a["wsb"], None)


@pytest.mark.parametrize("call", [norm, norm_backward])
def test_norm_refusals(b, call):
    r = lambda a, code, text: refused(b, call, a, code, text)  # noqa: E731
    new = lambda **k: change(b, norm_args(b), **k)  # noqa: E731
    F32, BF16 = b.GDP_F32, b.GDP_BF16
    r(new(x=None), b.GDP_EINVAL, "required")
    r(new(x=(BF16, [20, 192])), b.GDP_EINVAL, "x must be [T, G, V]")
    r(new(x=(b.GDP_I64, [20, 4, 48])), b.GDP_EUNSUPPORTED, "x must be float32")
    r(new(x=(BF16, [20, 0, 48])), b.GDP_EINVAL, "positive")
    r(new(x=(BF16, [20, 4, 16385])), b.GDP_EUNSUPPORTED, "16384")
    r(new(x=(BF16, [20, 65536, 48])), b.GDP_EUNSUPPORTED, "65535 groups")
    r(new(w=(F32, [47])), b.GDP_EINVAL, "weight: dim 0")
    r(new(w=(F32, [4, 4, 3])), b.GDP_EINVAL, "weight must be")
    r(new(w=(b.GDP_F16, [48])), b.GDP_EUNSUPPORTED, "weight must be")
    r(new(bias=(F32, [4, 48])), b.GDP_EINVAL, "share one shape")
    r(new(bias=(BF16, [48])), b.GDP_EINVAL, "share one shape")
    r(new(z=(F32, [20, 4, 48])), b.GDP_EUNSUPPORTED, "gate must have")
    r(new(z=(BF16, [20, 4, 47])), b.GDP_EINVAL, "gate: dim 2")
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        a = norm_args(b)
        a["eps"] = bad
        r(a, b.GDP_EINVAL, "eps")
    a = norm_args(b)
    a["act"] = 3
    r(a, b.GDP_EINVAL, "unknown activation")
    a = norm_args(b)
    a["x"].stride[1] = -48
    r(a, b.GDP_EINVAL, "negative strides")


def test_norm_output_refusals(b):
    new = lambda **k: change(b, norm_args(b), **k)  # noqa: E731
    refused(b, norm, new(y=None), b.GDP_EINVAL, "required")
    refused(b, norm, new(y=(b.GDP_F32, [20, 4, 48])), b.GDP_EUNSUPPORTED, "y must have")
    refused(b, norm, new(y=(b.GDP_BF16, [20, 4, 48], [192, 0, 1])), b.GDP_EALIAS, "its elements overlap")
    refused(b, norm, new(y=(b.GDP_BF16, [20, 4, 48], [100, 48, 1])), b.GDP_EALIAS, "its elements overlap")
    for other in ("x", "w", "bias", "z"):
        a = norm_args(b)
        a["y"].data = a[other].data
        refused(b, norm, a, b.GDP_EALIAS, "y overlaps input")


def test_norm_gradient_refusals(b):
    new = lambda **k: change(b, norm_args(b), **k)  # noqa: E731
    refused(b, norm_backward, new(dx=None), b.GDP_EINVAL, "required")
    refused(b, norm_backward, new(dw=None), b.GDP_EINVAL, "weight and dweight go together")
    refused(b, norm_backward, new(bias=None), b.GDP_EINVAL, "bias and dbias go together")
    refused(b, norm_backward, new(dz=None), b.GDP_EINVAL, "gate and dgate go together")
    refused(b, norm_backward, new(dw=(b.GDP_BF16, [48])), b.GDP_EUNSUPPORTED, "dweight must be float32")
    refused(b, norm_backward, new(db=(b.GDP_F32, [4, 48])), b.GDP_EINVAL, "dbias: expected 1 dims")
    refused(b, norm_backward, new(dy=(b.GDP_F32, [20, 4, 48])), b.GDP_EUNSUPPORTED, "d_y must have")
    for out in ("dx", "dz", "dw", "db"):
        for other in ("x", "dy", "z", "w", "bias"):
            a = norm_args(b)
            a[out].data = a[other].data
            refused(b, norm_backward, a, b.GDP_EALIAS, "overlaps input")
    a = norm_args(b)
    a["dz"].data = a["dx"].data
    refused(b, norm_backward, a, b.GDP_EALIAS, "overlaps")
    a = norm_args(b)
    a["wsb"] = 0
    refused(b, norm_backward, a, b.GDP_EWORKSPACE, "needed")
    for bad in ((-1, 1, 8), (1, 0, 8), (1, 1, 0), (1, 1, 16385)):
        assert b.gdp_group_norm_backward_workspace_bytes(*bad) == 0


def test_binding_refuses_host_tensors_and_unknown_names(b):
    x, g = torch.zeros(4, 8), torch.zeros(4, 8)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="on a GPU"):
        b.gated_scan(x, g, cu)
    with pytest.raises(ValueError, match="on a GPU"):
        b.gated_scan_decode(x, g, torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="on a GPU"):
        b.group_norm(torch.zeros(2, 2, 8))
    with pytest.raises(ValueError, match="activation must be one of"):
        b.group_norm(torch.zeros(2, 2, 8), activation="gelu")
