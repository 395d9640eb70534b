"""Refusals of the short convolution's, the selective scan's and the residual norm's entry points: host-side checks, no
GPU.  Pointers are fake, never dereferenced: every call here fails validation before a launch."""
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


def refused(b, call, a, code, fragment):
    assert call(b, a) == code, b.gdp_last_error()
    assert fragment in b.gdp_last_error(), b.gdp_last_error()


def change(b, a, **new):
    """a with tensors replaced: name=(dtype, shape[, strides]), or None for absent."""
    for k, v in new.items():
        a[k] = None if v is None else a["fake"].tensor(b, *v)
    return a


# ------------------------------------------------------------ short convolution

def conv_args(b, T=200, N=3, D=96, W=4, dt=None):
    f = Fake()
    dt = b.GDP_BF16 if dt is None else dt
    F32 = b.GDP_F32
    a = dict(x=f.tensor(b, dt, [T, D]), w=f.tensor(b, F32, [D, W]), bc=f.tensor(b, F32, [D]), act=1,
             cu=f.tensor(b, b.GDP_I32, [N + 1]), s0=f.tensor(b, dt, [N, W - 1, D]), ofs=1,
             cache=f.tensor(b, dt, [5, W - 1, D]), slots=f.tensor(b, b.GDP_I32, [N]), y=f.tensor(b, dt, [T, D]),
             fs=f.tensor(b, dt, [N, W - 1, D]), dy=f.tensor(b, dt, [T, D]), df=f.tensor(b, F32, [N, W - 1, D]),
             dx=f.tensor(b, dt, [T, D]), dw=f.tensor(b, F32, [D, W]), db=f.tensor(b, F32, [D]),
             ds0=f.tensor(b, F32, [N, W - 1, D]), ws=f.next, wsb=1 << 28, fake=f)
    f.next += 1 << 30
    return a


def conv(b, a):
    return b.LIB.gdp_short_conv(ref(a["x"]), ref(a["w"]), ref(a["bc"]), a["act"], ref(a["cu"]), ref(a["s0"]), a["ofs"],
                                ref(a["cache"]), ref(a["slots"]), ref(a["y"]), ref(a["fs"]), None)


def conv_backward(b, a):
    return b.LIB.gdp_short_conv_backward(ref(a["x"]), ref(a["w"]), ref(a["bc"]), a["act"], ref(a["cu"]), ref(a["s0"]),
                                         ref(a["dy"]), ref(a["df"]), ref(a["dx"]), ref(a["dw"]), ref(a["db"]),
                                         ref(a["ds0"]), a["ws"], a["wsb"], None)


def conv_decode(b, a):
    return b.LIB.gdp_short_conv_decode(ref(a["x"]), ref(a["w"]), ref(a["bc"]), a["act"], ref(a["cache"]),
                                       ref(a["slots"]), ref(a["y"]), None)


@pytest.mark.parametrize("call", [conv, conv_backward])
def test_conv_operands(b, call):
    E, U = b.GDP_EINVAL, b.GDP_EUNSUPPORTED
    args = lambda **new: change(b, conv_args(b), **new)  # noqa: E731
    refused(b, call, args(x=None), E, "required")
    refused(b, call, args(w=None), E, "required")
    refused(b, call, args(cu=None), E, "cu_seqlens is required")
    refused(b, call, args(x=(b.GDP_BF16, [200, 4, 24])), E, "x must be [T, D]")
    refused(b, call, args(x=(b.GDP_BF16, [200, 0])), E, "at least one channel")
    refused(b, call, args(x=(b.GDP_I32, [200, 96])), U, "x must be float32")
    refused(b, call, args(w=(b.GDP_F32, [96])), E, "weight must be [D, W]")
    refused(b, call, args(w=(b.GDP_F32, [95, 4])), E, "weight: dim 0")
    refused(b, call, args(w=(b.GDP_F32, [96, 1])), U, "2 to 8 taps")
    refused(b, call, args(w=(b.GDP_F32, [96, 9])), U, "2 to 8 taps")
    refused(b, call, args(w=(b.GDP_F32, [96, 4], [8, 1])), E, "weight must be contiguous")
    refused(b, call, args(w=(b.GDP_F16, [96, 4])), U, "weight must be float32")
    refused(b, call, args(bc=(b.GDP_BF16, [96])), E, "share one dtype")
    refused(b, call, args(bc=(b.GDP_F32, [97])), E, "bias: dim 0")
    refused(b, call, args(cu=(b.GDP_F32, [4])), E, "int32 or int64")
    refused(b, call, args(s0=(b.GDP_F32, [3, 3, 96])), U, "initial_state must be of the input's dtype")
    refused(b, call, args(s0=(b.GDP_BF16, [3, 96, 3])), E, "initial_state: dim 1")
    refused(b, call, args(s0=(b.GDP_BF16, [3, 3, 96], [400, 96, 1])), E, "initial_state must be contiguous")
    a = conv_args(b)
    a["act"] = 7
    refused(b, call, a, E, "unknown activation")
    a = conv_args(b)
    a["x"].stride[0] = -96
    refused(b, call, a, E, "negative strides")
    a = conv_args(b)
    a["x"].shape[0] = (1 << 30) + 1
    refused(b, call, a, U, "launch limits")


def test_conv_outputs(b):
    E, U = b.GDP_EINVAL, b.GDP_EUNSUPPORTED
    args = lambda **new: change(b, conv_args(b), **new)  # noqa: E731
    refused(b, conv, args(y=None), E, "y is required")
    refused(b, conv, args(y=(b.GDP_F32, [200, 96])), U, "y must have x's dtype")
    refused(b, conv, args(y=(b.GDP_BF16, [200, 96], [95, 1])), b.GDP_EALIAS, "rows overlap")
    refused(b, conv, args(fs=None), E, "output_final_state needs")
    refused(b, conv, args(slots=None), E, "go together")
    refused(b, conv, args(cache=None), E, "go together")
    refused(b, conv, args(cache=(b.GDP_F32, [5, 3, 96])), U, "state_cache must be of the input's dtype")
    refused(b, conv, args(slots=(b.GDP_I32, [4])), E, "state_indices: dim 0")
    refused(b, conv, args(slots=(b.GDP_F32, [3])), E, "state_indices must be")
    for out in ("y", "fs", "cache"):
        for other in ("x", "w", "bc", "cu", "s0", "slots"):
            a = conv_args(b)
            a[out].data = a[other].data
            refused(b, conv, a, b.GDP_EALIAS, "overlaps input")
    a = conv_args(b)
    a["fs"].data = a["cache"].data
    refused(b, conv, a, b.GDP_EALIAS, "overlaps")


def test_conv_step(b):
    E, U = b.GDP_EINVAL, b.GDP_EUNSUPPORTED
    args = lambda **new: change(b, {**conv_args(b, T=3), **{}}, **new)  # noqa: E731
    refused(b, conv_decode, args(cache=None), E, "required")
    refused(b, conv_decode, args(slots=None), E, "required")
    refused(b, conv_decode, args(cache=(b.GDP_BF16, [5, 4, 96])), E, "state_cache: dim 1")
    refused(b, conv_decode, args(slots=(b.GDP_I64, [2])), E, "state_indices: dim 0")
    refused(b, conv_decode, args(y=(b.GDP_F16, [3, 96])), U, "y must have")
    for out in ("y", "cache"):
        for other in ("x", "w", "bc", "slots"):
            a = args()
            a[out].data = a[other].data
            refused(b, conv_decode, a, b.GDP_EALIAS, "overlaps input")


def test_conv_gradients(b):
    E, U = b.GDP_EINVAL, b.GDP_EUNSUPPORTED
    args = lambda **new: change(b, conv_args(b), **new)  # noqa: E731
    for k in ("dy", "dx", "dw"):
        refused(b, conv_backward, args(**{k: None}), E, "required")
    refused(b, conv_backward, args(db=None), E, "go together")
    refused(b, conv_backward, args(bc=None), E, "go together")
    refused(b, conv_backward, args(dx=(b.GDP_F32, [200, 96])), U, "dx must have x's dtype")
    refused(b, conv_backward, args(dw=(b.GDP_BF16, [96, 4])), U, "dweight must be float32")
    refused(b, conv_backward, args(df=(b.GDP_BF16, [3, 3, 96])), U, "d_final_state must be float32")
    refused(b, conv_backward, args(ds0=(b.GDP_F32, [3, 3, 95])), E, "d_initial_state: dim 2")
    for out in ("dx", "dw", "db", "ds0"):
        for other in ("x", "w", "bc", "cu", "s0", "dy", "df"):
            a = conv_args(b)
            a[out].data = a[other].data
            refused(b, conv_backward, a, b.GDP_EALIAS, "overlaps input")
    need = b.gdp_short_conv_backward_workspace_bytes(200, 3, 96, 4)
    for new in ({"ws": None}, {"wsb": need - 1}):
        refused(b, conv_backward, {**conv_args(b), **new}, b.GDP_EWORKSPACE, "workspace of")
    a = conv_args(b)
    a["ws"] += 128
    refused(b, conv_backward, a, b.GDP_EWORKSPACE, "256-byte")
    a = conv_args(b)
    a["dx"].data = a["ws"]
    refused(b, conv_backward, a, b.GDP_EALIAS, "workspace")
    for bad in ((-1, 3, 96, 4), (200, -1, 96, 4), (200, 3, 0, 4), (200, 3, 96, 1), (200, 3, 96, 9), (1 << 31, 3, 96, 4)):
        assert b.gdp_short_conv_backward_workspace_bytes(*bad) == 0


# --------------------------------------------------------------- selective scan

def select_args(b, T=200, N=3, D=96, G=2, S=16, dt=None):
    f = Fake()
    dt = b.GDP_BF16 if dt is None else dt
    F32 = b.GDP_F32
    a = dict(u=f.tensor(b, dt, [T, D]), dt=f.tensor(b, F32, [T, D]), A=f.tensor(b, F32, [D, S]),
             B=f.tensor(b, dt, [T, G, S]), C=f.tensor(b, dt, [T, G, S]), skip=f.tensor(b, F32, [D]),
             z=f.tensor(b, dt, [T, D]), bias=f.tensor(b, F32, [D]), sp=1, cu=f.tensor(b, b.GDP_I32, [N + 1]),
             s0=f.tensor(b, F32, [N, D, S]), ofs=1, cache=f.tensor(b, F32, [5, D, S]),
             slots=f.tensor(b, b.GDP_I32, [N]), rcp=1, o=f.tensor(b, dt, [T, D]), fs=f.tensor(b, F32, [N, D, S]),
             cp=f.tensor(b, F32, [T // 16 + N, S, D]), do=f.tensor(b, dt, [T, D]), df=f.tensor(b, F32, [N, D, S]),
             du=f.tensor(b, dt, [T, D]), ddt=f.tensor(b, F32, [T, D]), dA=f.tensor(b, F32, [D, S]),
             dB=f.tensor(b, dt, [T, G, S]), dC=f.tensor(b, dt, [T, G, S]), dskip=f.tensor(b, F32, [D]),
             dz=f.tensor(b, dt, [T, D]), dbias=f.tensor(b, F32, [D]), ds0=f.tensor(b, F32, [N, D, S]), ws=f.next,
             wsb=1 << 28, fake=f)
    f.next += 1 << 30
    return a


INS = ("u", "dt", "A", "B", "C", "skip", "z", "bias")


def select(b, a):
    return b.LIB.gdp_selective_scan(*[ref(a[k]) for k in INS], a["sp"], ref(a["cu"]), ref(a["s0"]), a["ofs"],
                                    ref(a["cache"]), ref(a["slots"]), a["rcp"], ref(a["o"]), ref(a["fs"]),
                                    ref(a["cp"]), a["ws"], a["wsb"], None)


def select_decode(b, a):
    return b.LIB.gdp_selective_scan_decode(*[ref(a[k]) for k in INS], a["sp"], ref(a["cache"]), ref(a["slots"]),
                                           ref(a["o"]), None)


def select_backward(b, a):
    outs = ("cp", "do", "df", "du", "ddt", "dA", "dB", "dC", "dskip", "dz", "dbias", "ds0")
    return b.LIB.gdp_selective_scan_backward(*[ref(a[k]) for k in INS], a["sp"], ref(a["cu"]), ref(a["s0"]),
                                             *[ref(a[k]) for k in outs], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("call", [select, select_backward, select_decode])
def test_select_operands(b, call):
    E, U = b.GDP_EINVAL, b.GDP_EUNSUPPORTED
    T = 3 if call is select_decode else 200
    args = lambda **new: change(b, select_args(b, T=T), **new)  # noqa: E731
    for k in ("u", "dt", "A", "B", "C"):
        refused(b, call, args(**{k: None}), E, "required")
    refused(b, call, args(u=(b.GDP_BF16, [T, 4, 24])), E, "u must be [T, D]")
    refused(b, call, args(u=(b.GDP_BF16, [T, 0])), E, "at least one channel")
    refused(b, call, args(u=(b.GDP_I64, [T, 96])), U, "u must be float32")
    refused(b, call, args(dt=(b.GDP_F16, [T, 96])), U, "dt must be float32 or")
    refused(b, call, args(dt=(b.GDP_F32, [T, 95])), E, "dt: dim 1")
    refused(b, call, args(A=(b.GDP_F32, [96])), E, "A must be [D, S]")
    refused(b, call, args(A=(b.GDP_BF16, [96, 16])), U, "A must be float32")
    refused(b, call, args(A=(b.GDP_F32, [96, 33])), U, "1 to 32 states")
    refused(b, call, args(A=(b.GDP_F32, [96, 0])), U, "1 to 32 states")
    refused(b, call, args(A=(b.GDP_F32, [96, 16], [20, 1])), E, "A must be contiguous")
    refused(b, call, args(B=(b.GDP_BF16, [T, 32])), E, "B must be [T, G, S]")
    refused(b, call, args(B=(b.GDP_F32, [T, 2, 16])), U, "B and C must have")
    refused(b, call, args(B=(b.GDP_BF16, [T, 5, 16])), E, "a multiple of the 5 groups")
    refused(b, call, args(C=(b.GDP_BF16, [T, 2, 15])), E, "C: dim 2")
    refused(b, call, args(C=(b.GDP_BF16, [T, 2, 16], [64, 32, 2])), E, "innermost")
    refused(b, call, args(skip=(b.GDP_BF16, [96])), U, "skip must be float32")
    refused(b, call, args(bias=(b.GDP_F32, [95])), E, "dt_bias: dim 0")
    refused(b, call, args(z=(b.GDP_F32, [T, 96])), U, "gate must have")
    for k in ("u", "B"):
        a = args()
        a[k].stride[0] = -1
        refused(b, call, a, E, "negative strides")


@pytest.mark.parametrize("call", [select, select_backward])
def test_select_sequences(b, call):
    E, U = b.GDP_EINVAL, b.GDP_EUNSUPPORTED
    args = lambda **new: change(b, select_args(b), **new)  # noqa: E731
    refused(b, call, args(cu=None), E, "cu_seqlens is required")
    refused(b, call, args(cu=(b.GDP_I32, [2, 2])), E, "cu_seqlens must be a contiguous")
    refused(b, call, args(s0=(b.GDP_F32, [3, 16, 96])), E, "initial_state: dim 1")
    refused(b, call, args(s0=(b.GDP_BF16, [3, 96, 16])), U, "initial_state must be float32")
    refused(b, call, args(cp=(b.GDP_F32, [14, 16, 96])), E, "checkpoints: dim 0")
    need = (b.gdp_selective_scan_workspace_bytes(200, 3, 96, 2, 16) if call is select else
            b.gdp_selective_scan_backward_workspace_bytes(200, 3, 96, 2, 16, True))
    for new in ({"ws": None}, {"wsb": need - 1}):
        refused(b, call, {**select_args(b), **new}, b.GDP_EWORKSPACE, "workspace of")
    a = select_args(b)
    a["ws"] += 128
    refused(b, call, a, b.GDP_EWORKSPACE, "256-byte")
    outs = ("o", "fs", "cache", "cp") if call is select else ("du", "ddt", "dA", "dB", "dC", "dskip", "dz", "dbias", "ds0")
    others = INS + ("cu", "s0") + (("slots",) if call is select else ("cp", "do", "df"))
    for out in outs:
        for other in others:
            a = select_args(b)
            a[out].data = a[other].data
            refused(b, call, a, b.GDP_EALIAS, "overlaps input")
        a = select_args(b)
        a[out].data = a["ws"]
        refused(b, call, a, b.GDP_EALIAS, "workspace")


def test_select_outputs(b):
    E, U = b.GDP_EINVAL, b.GDP_EUNSUPPORTED
    args = lambda **new: change(b, select_args(b), **new)  # noqa: E731
    refused(b, select, args(o=None), E, "o is required")
    refused(b, select, args(o=(b.GDP_F32, [200, 96])), U, "o must have u's dtype")
    refused(b, select, args(fs=None), E, "output_final_state needs")
    refused(b, select, args(cp=None), E, "return_checkpoints needs")
    refused(b, select, args(slots=None), E, "go together")
    refused(b, select, args(cache=(b.GDP_F32, [5, 16, 96])), E, "state_cache: dim 1")
    refused(b, select, args(slots=(b.GDP_I32, [2])), E, "state_indices: dim 0")
    for k in ("du", "ddt", "dA", "dB", "dC"):
        refused(b, select_backward, args(**{k: None}), E, "required")
    for k in ("skip", "z", "bias", "dskip", "dz", "dbias"):
        refused(b, select_backward, args(**{k: None}), E, "go together")
    refused(b, select_backward, args(do=None), E, "d_o is required")
    refused(b, select_backward, args(do=(b.GDP_F32, [200, 96])), U, "share one dtype")
    refused(b, select_backward, args(du=(b.GDP_F32, [200, 96])), U, "du must have u's dtype")
    refused(b, select_backward, args(ddt=(b.GDP_BF16, [200, 96])), U, "ddt must have dt's dtype")
    refused(b, select_backward, args(dB=(b.GDP_F32, [200, 2, 16])), U, "dB must be")
    refused(b, select_backward, args(dC=(b.GDP_BF16, [200, 2, 16], [64, 16, 1])), E, "dC must be contiguous")
    refused(b, select_backward, args(ds0=(b.GDP_F32, [3, 96, 15])), E, "d_initial_state: dim 2")
    # without checkpoints the workspace has room for them
    a = change(b, select_args(b), cp=None)
    a["wsb"] = b.gdp_selective_scan_backward_workspace_bytes(200, 3, 96, 2, 16, True)
    refused(b, select_backward, a, b.GDP_EWORKSPACE, "workspace of")
    step = lambda **new: change(b, select_args(b, T=3), **new)  # noqa: E731
    refused(b, select_decode, step(cache=None), E, "required")
    refused(b, select_decode, step(slots=(b.GDP_I32, [4])), E, "state_indices: dim 0")
    for out in ("o", "cache"):
        for other in INS + ("slots",):
            a = step()
            a[out].data = a[other].data
            refused(b, select_decode, a, b.GDP_EALIAS, "overlaps input")
    for bad in ((-1, 3, 96, 2, 16), (200, -1, 96, 2, 16), (200, 3, 96, 5, 16), (200, 3, 96, 2, 33), (200, 3, 96, 0, 16)):
        assert b.gdp_selective_scan_workspace_bytes(*bad) == 0
        assert b.gdp_selective_scan_backward_workspace_bytes(*bad, False) == 0


# ---------------------------------------------------------- norms around a block

def norm_args(b, T=20, D=96, dt=None, stream=None):
    f = Fake()
    dt = b.GDP_BF16 if dt is None else dt
    st = b.GDP_F32 if stream is None else stream
    F32 = b.GDP_F32
    a = dict(x=f.tensor(b, st, [T, D]), y=f.tensor(b, dt, [T, D]), wa=f.tensor(b, F32, [D]), wb=f.tensor(b, F32, [D]),
             z=f.tensor(b, dt, [T, D]), act=2, post=1, pre=1, scale=0.5, eps=1e-5, r=f.tensor(b, st, [T, D]),
             n=f.tensor(b, dt, [T, D]), dr=f.tensor(b, st, [T, D]), dn=f.tensor(b, dt, [T, D]),
             dx=f.tensor(b, st, [T, D]), dy=f.tensor(b, dt, [T, D]), dwa=f.tensor(b, F32, [D]),
             dwb=f.tensor(b, F32, [D]), dz=f.tensor(b, dt, [T, D]), ws=f.next, wsb=1 << 28, fake=f)
    f.next += 1 << 30
    return a


def norm(b, a):
    return b.LIB.gdp_residual_norm(ref(a["x"]), ref(a["y"]), ref(a["wa"]), ref(a["wb"]), ref(a["z"]), a["act"],
                                   a["post"], a["pre"], a["scale"], a["eps"], ref(a["r"]), ref(a["n"]), None)


def norm_backward(b, a):
    return b.LIB.gdp_residual_norm_backward(ref(a["x"]), ref(a["y"]), ref(a["wa"]), ref(a["wb"]), ref(a["z"]), a["act"],
                                            a["post"], a["pre"], a["scale"], a["eps"], ref(a["dr"]), ref(a["dn"]),
                                            ref(a["dx"]), ref(a["dy"]), ref(a["dwa"]), ref(a["dwb"]), ref(a["dz"]),
                                            a["ws"], a["wsb"], None)


@pytest.mark.parametrize("call", [norm, norm_backward])
def test_norm_operands(b, call):
    E, U = b.GDP_EINVAL, b.GDP_EUNSUPPORTED
    args = lambda **new: change(b, norm_args(b), **new)  # noqa: E731
    refused(b, call, args(x=None), E, "required")
    refused(b, call, args(y=None), E, "required")
    refused(b, call, args(y=(b.GDP_BF16, [20, 2, 48])), E, "y must be [T, D]")
    refused(b, call, args(y=(b.GDP_BF16, [20, 0])), E, "at least one channel")
    refused(b, call, args(y=(b.GDP_I32, [20, 96])), U, "y must be float32")
    refused(b, call, args(x=(b.GDP_F16, [20, 96])), U, "x must be float32 or")
    refused(b, call, args(x=(b.GDP_F32, [19, 96])), E, "x: dim 0")
    refused(b, call, args(y=(b.GDP_BF16, [20, 16385])), U, "more than 16384 channels")
    refused(b, call, args(wa=(b.GDP_F16, [96])), U, "post_weight must be float32 or")
    refused(b, call, args(wb=(b.GDP_BF16, [96])), E, "share one dtype")
    refused(b, call, args(wb=(b.GDP_F32, [95])), E, "pre_weight: dim 0")
    refused(b, call, args(z=(b.GDP_F32, [20, 96])), U, "gate must have")
    refused(b, call, args(z=None), E, "an activation needs a gate")
    for k, v, text in (("act", 3, "unknown activation"), ("eps", 0.0, "eps must be"), ("eps", float("nan"), "eps must be"),
                       ("eps", 1e-39, "eps must be"), ("eps", float("inf"), "eps must be"),
                       ("scale", float("inf"), "residual_scale must be finite"), ("pre", 0, "pre_weight needs pre_norm")):
        refused(b, call, {**norm_args(b), k: v}, E, text)
    a = args()
    a["y"].stride[0] = -96
    refused(b, call, a, E, "negative strides")


def test_norm_outputs(b):
    E, U = b.GDP_EINVAL, b.GDP_EUNSUPPORTED
    args = lambda **new: change(b, norm_args(b), **new)  # noqa: E731
    refused(b, norm, args(r=None), E, "r is required")
    refused(b, norm, args(n=None), E, "go together")
    a = change(b, norm_args(b), wb=None)
    a["pre"] = 0
    refused(b, norm, a, E, "go together")
    refused(b, norm, args(r=(b.GDP_BF16, [20, 96])), U, "r must have x's dtype")
    refused(b, norm, args(n=(b.GDP_F32, [20, 96])), U, "n must have y's dtype")
    refused(b, norm, args(r=(b.GDP_F32, [20, 96], [64, 1])), b.GDP_EALIAS, "rows overlap")
    for out, others in (("r", ("y", "wa", "wb", "z")), ("n", ("x", "y", "wa", "wb", "z"))):
        for other in others:
            a = args()
            a[out].data = a[other].data
            refused(b, norm, a, b.GDP_EALIAS, "overlaps input")
    # x in place: that view and no other one, and n still apart
    a = args()
    a["r"].data = a["x"].data + 4
    refused(b, norm, a, b.GDP_EALIAS, "r overlaps input x")
    a = args(r=(b.GDP_F32, [20, 96], [192, 1]))
    a["r"].data = a["x"].data
    refused(b, norm, a, b.GDP_EALIAS, "r overlaps input x")
    a = args()
    a["r"].data = a["n"].data = a["x"].data
    refused(b, norm, a, b.GDP_EALIAS, "r overlaps n")
    a = args(x=(b.GDP_F32, [20, 96], [0, 1]))
    a["r"].data = a["x"].data
    refused(b, norm, a, b.GDP_EALIAS, "r overlaps input x")


def test_norm_gradients(b):
    E, U = b.GDP_EINVAL, b.GDP_EUNSUPPORTED
    args = lambda **new: change(b, norm_args(b), **new)  # noqa: E731
    for k in ("dx", "dy"):
        refused(b, norm_backward, args(**{k: None}), E, "required")
    for k in ("dwa", "dwb", "dz", "wa", "wb", "dn"):
        refused(b, norm_backward, args(**{k: None}), E, "go together")
    a = change(b, norm_args(b), wb=None, dwb=None, dn=None, dr=None)
    a["pre"] = 0
    refused(b, norm_backward, a, E, "d_r is required")
    refused(b, norm_backward, args(dr=(b.GDP_BF16, [20, 96])), U, "d_r must have x's dtype")
    refused(b, norm_backward, args(dn=(b.GDP_F32, [20, 96])), U, "d_n must have y's dtype")
    refused(b, norm_backward, args(dy=(b.GDP_F32, [20, 96])), U, "dy must have y's dtype")
    refused(b, norm_backward, args(dwa=(b.GDP_BF16, [96])), U, "dpost_weight must be float32")
    for out in ("dx", "dy", "dwa", "dwb", "dz"):
        for other in ("x", "y", "wa", "wb", "z", "dr", "dn"):
            a = args()
            a[out].data = a[other].data
            refused(b, norm_backward, a, b.GDP_EALIAS, "overlaps input")
    need = b.gdp_residual_norm_backward_workspace_bytes(20, 96)
    for new in ({"ws": None}, {"wsb": need - 1}):
        refused(b, norm_backward, {**norm_args(b), **new}, b.GDP_EWORKSPACE, "workspace of")
    for bad in ((-1, 96), (20, 0), (20, 16385)):
        assert b.gdp_residual_norm_backward_workspace_bytes(*bad) == 0


# ------------------------------------------------------------------- front ends

def test_front_ends_refuse_host_tensors_and_names(b):
    x, w, cu = torch.zeros(4, 8), torch.zeros(8, 4), torch.tensor([0, 4])
    A, B = torch.zeros(8, 2), torch.zeros(4, 1, 2)
    for call in (lambda: b.short_conv(x, w, cu), lambda: b.short_conv_backward(x, w, cu, x),
                 lambda: b.short_conv_decode(x, w, torch.zeros(4, 3, 8), cu.new_zeros(4)),
                 lambda: b.selective_scan(x, x, A, B, B, cu), lambda: b.selective_scan_backward(x, x, A, B, B, cu, x),
                 lambda: b.selective_scan_decode(x, x, A, B, B, torch.zeros(4, 8, 2), cu.new_zeros(4)),
                 lambda: b.residual_norm(x, x), lambda: b.residual_norm_backward(x, x, x, x)):
        with pytest.raises(ValueError, match="on a GPU"):
            call()
    with pytest.raises(ValueError, match="activation must be"):
        b.short_conv(x, w, cu, activation="tanh")
    with pytest.raises(ValueError, match="activation must be"):
        b.residual_norm(x, x, gate=x, activation="gelu")
