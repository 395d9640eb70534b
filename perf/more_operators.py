"""Measured cases of the short causal convolution, of the selective state space scan and of the norms around a block.

Each case is one call (or one training step) of

    y_t = act(b + sum_j w_j x_{t-W+1+j}),                           per channel over packed sequences,

    h_t = exp(delta_t A) h_{t-1} + delta_t u_t B_t,   delta = softplus(dt + dt_bias),
    o_t = (C_t . h_t + skip u_t) silu(gate_t),                      N states per channel,

    r = x + s act(gate) norm(y) w_post,   n = norm(r) w_pre,        per token over all channels,

of the first two's single-token step on a state cache, or of the gradients, in
the plain form below (elementary torch operations in 32 bits, rounded once at
the end) or, where `own` is set, through the library's binding.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5


# ------------------------------------------------------------------- cases

def _serving_lengths(most):
    """64 prompt lengths spread over 1..most and four empty padding entries (the serving mix's shape)."""
    return ",".join(str(1 + (i * 2531 + 977) % most) for i in range(64)) + ",0,0,0,0"


def listed():
    return [
        # the smallest prompt batch: queries, keys and values of 4 heads x 128, carried state in and out (latency)
        {"name": "conv_prompts", "op": "conv", "lens": "37,64,200,511", "D": 1536, "W": 4, "dtype": "bf16",
         "bias": False, "act": "silu", "initial": True, "slots": 0},
        # a serving step's prompts, 32 heads x 128, the last inputs into the slots of a state cache
        {"name": "conv_serving", "op": "conv", "lens": _serving_lengths(4096), "D": 4096, "W": 4, "dtype": "bf16",
         "bias": True, "act": "silu", "initial": False, "slots": 128},
        # a training step in float32 over ragged lengths, a channel count no vector width divides, states carried
        {"name": "conv_train_ragged", "op": "conv_train", "lens": "1,1023,77,0,2500,640,3,4001", "D": 1001, "W": 3,
         "dtype": "f32", "bias": True, "act": "silu", "initial": True},
        # a full serving batch's next tokens, some entries padding
        {"name": "conv_step", "op": "conv_decode", "N": 256, "D": 4096, "W": 4, "slots": 1024, "pad": 8,
         "dtype": "bf16", "bias": True, "act": "silu"},
        # the smallest prompt batch through 512 channels of 16 states, carried state in and out (latency)
        {"name": "select_prompts", "op": "select", "lens": "37,64,200,511", "D": 512, "S": 16, "G": 1,
         "dtype": "bf16", "dt": "bf16", "gated": True, "initial": True, "slots": 0},
        # one long document: few channels, a long time axis
        {"name": "select_document", "op": "select", "lens": "32768", "D": 2048, "S": 16, "G": 1, "dtype": "bf16",
         "dt": "f32", "gated": True, "initial": False, "slots": 0},
        # a serving step's prompts, final states into the slots of a state cache
        {"name": "select_serving", "op": "select", "lens": _serving_lengths(1024), "D": 4096, "S": 16, "G": 1,
         "dtype": "bf16", "dt": "bf16", "gated": True, "initial": False, "slots": 128},
        # a training step's forward and backward pass over equal sequences
        {"name": "select_train", "op": "select_train", "lens": "2048,2048,2048,2048", "D": 2048, "S": 16, "G": 1,
         "dtype": "bf16", "dt": "bf16", "gated": True, "initial": False},
        # a full serving batch's next tokens, some entries padding
        {"name": "select_step", "op": "select_decode", "N": 256, "D": 4096, "S": 16, "G": 1, "slots": 1024, "pad": 8,
         "dtype": "bf16", "dt": "bf16", "gated": True},
        # the norms between two blocks at one decoded token (latency)
        {"name": "between_token", "op": "between", "T": 1, "D": 4096, "dtype": "bf16", "stream": "bf16",
         "post": True, "pre": True, "gated": True, "act": "sigmoid", "scale": 0.5},
        # the same after a long prefill, without a gate
        {"name": "between_prefill", "op": "between", "T": 65536, "D": 4096, "dtype": "bf16", "stream": "bf16",
         "post": True, "pre": True, "gated": False, "act": "none", "scale": 1.0},
        # a training step of them with a float32 residual stream, an odd number of tokens
        {"name": "between_train", "op": "between_train", "T": 8195, "D": 4096, "dtype": "f16", "stream": "f32",
         "post": True, "pre": True, "gated": True, "act": "sigmoid", "scale": 0.25},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_lens(rng, tokens):
    count = min(_log_int(rng, 1, 64), tokens)
    cuts = sorted(rng.randint(0, tokens) for _ in range(count - 1))
    edges = [0] + cuts + [tokens]
    return ",".join(str(b - a) for a, b in zip(edges, edges[1:]))


def _draw_channels(rng, hi, groups=1):
    step = rng.choice([64, 64, 8, 1]) * groups
    return max(step, _log_int(rng, 64, hi) // step * step)


def draw(rng):
    op = rng.choice(["conv", "conv_train", "conv_decode", "select", "select", "select_train", "select_decode",
                     "between", "between_train"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("conv", "conv_train", "conv_decode"):
        form = {"op": op, "D": _draw_channels(rng, 4096), "W": rng.choice([2, 3, 4, 4, 4, 6, 8]), "dtype": dtype,
                "bias": flag(), "act": rng.choice(["none", "silu", "silu", "sigmoid"])}
        if op == "conv_decode":
            N = _log_int(rng, 1, 512)
            return {**form, "N": N, "slots": 1024, "pad": rng.randint(0, N // 8)}
        tokens = _log_int(rng, 64, 65536 if op == "conv" else 32768)
        form.update(lens=_draw_lens(rng, tokens), initial=flag())
        return {**form, "slots": 128 if flag() else 0} if op == "conv" else form
    if op in ("select", "select_train", "select_decode"):
        G = rng.choice([1, 1, 1, 2, 4])
        form = {"op": op, "S": rng.choice([16, 16, 16, 8, 32, 5]), "G": G, "dtype": dtype,
                "dt": rng.choice(["f32", dtype]), "gated": flag()}
        if op == "select_decode":
            N = _log_int(rng, 1, 512)
            return {**form, "N": N, "D": _draw_channels(rng, 4096, G), "slots": 1024, "pad": rng.randint(0, N // 8)}
        # 32 states cost twice what 16 do
        many = 2 if form["S"] > 16 else 1
        D = _draw_channels(rng, (4096 if op == "select" else 2048) // many, G)
        tokens = _log_int(rng, 64, 32768 if op == "select" else 8192)
        form.update(D=D, lens=_draw_lens(rng, tokens), initial=flag())
        return {**form, "slots": 128 if flag() else 0} if op == "select" else form
    gated = flag()
    return {"op": op, "T": _log_int(rng, 1, 32768 if op == "between" else 16384), "D": _draw_channels(rng, 4096),
            "dtype": dtype, "stream": rng.choice(["f32", dtype]), "post": flag(), "pre": rng.random() < 0.8,
            "gated": gated, "act": rng.choice(["none", "sigmoid", "silu"]) if gated else "none",
            "scale": rng.choice([1.0, 0.5, 0.125])}


# ------------------------------------------------------------------ inputs

def _lens(case):
    return [int(s) for s in case["lens"].split(",")]


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=gen.device, dtype=torch.float32)


def _rand(gen, *shape):
    return torch.rand(*shape, generator=gen, device=gen.device, dtype=torch.float32)


def _packed(s, case):
    """cu_seqlens of the case's lengths, and slots of the cache: padding entries have none."""
    lens = torch.tensor([0] + _lens(case))
    s["cu"] = lens.cumsum(0).to(torch.int32).cuda()
    return int(lens.sum()), len(lens) - 1


def _slots(s, gen, count, N, pad=0):
    slots = torch.randperm(count, generator=gen, device="cuda")[:N]
    if "cu" in s:
        slots = torch.where(s["cu"][1:] == s["cu"][:-1], -1, slots)
    slots[:pad] = -1
    s["slots"] = slots.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    op, D = case["op"], case["D"]
    s = {"case": dict(case), "cache": None, "slots": None}
    train = op.endswith("_train")
    if op in ("conv", "conv_train", "conv_decode"):
        W = case["W"]
        s["w"] = (_rand(gen, D, W) * 2 - 1) / math.sqrt(W)
        s["b"] = 0.1 * _randn(gen, D) if case["bias"] else None
        T, N = (case["N"], case["N"]) if op == "conv_decode" else _packed(s, case)
        s["x"] = _randn(gen, T, D).to(dt)
        if op != "conv_decode":
            s["s0"] = _randn(gen, N, W - 1, D).to(dt) if case["initial"] else None
        if case.get("slots"):
            s["cache"] = _randn(gen, case["slots"], W - 1, D).to(dt)
            _slots(s, gen, case["slots"], N, case.get("pad", 0))
        if train:
            s["d_y"] = _randn(gen, T, D).to(dt)
            s["d_final"] = _randn(gen, N, W - 1, D) if case["initial"] else None
    elif op in ("select", "select_train", "select_decode"):
        S, G = case["S"], case["G"]
        # -A = 1 .. S, scattered a little; steps of 0.001 to 0.1 before what the input adds to them
        s["A"] = -torch.arange(1, S + 1, device="cuda") * (0.1 * _randn(gen, D, S)).exp()
        step = (math.log(0.001) + _rand(gen, D) * math.log(100.0)).exp()
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["skip"] = 1.0 + 0.1 * _randn(gen, D)
        T, N = (case["N"], case["N"]) if op == "select_decode" else _packed(s, case)
        s["u"] = _randn(gen, T, D).to(dt)
        s["dt"] = _randn(gen, T, D).to(DTYPES[case["dt"]])
        s["B"], s["C"] = _randn(gen, T, G, S).to(dt), _randn(gen, T, G, S).to(dt)
        s["z"] = _randn(gen, T, D).to(dt) if case["gated"] else None
        if op != "select_decode":
            s["s0"] = 0.1 * _randn(gen, N, D, S) if case["initial"] else None
        if case.get("slots"):
            s["cache"] = 0.1 * _randn(gen, case["slots"], D, S)
            _slots(s, gen, case["slots"], N, case.get("pad", 0))
        if train:
            s["d_o"] = _randn(gen, T, D).to(dt)
            s["d_final"] = _randn(gen, N, D, S) if case["initial"] else None
    else:
        T, stream = case["T"], DTYPES[case["stream"]]
        s["x"] = _randn(gen, T, D).to(stream)
        s["y"] = (0.5 * _randn(gen, T, D)).to(dt)
        s["z"] = _randn(gen, T, D).to(dt) if case["gated"] else None
        s["w_post"] = 1.0 + 0.1 * _randn(gen, D)
        s["w_pre"] = 1.0 + 0.1 * _randn(gen, D) if case["pre"] else None
        if train:
            s["d_r"] = _randn(gen, T, D).to(stream)
            s["d_n"] = _randn(gen, T, D).to(dt) if case["pre"] else None
    return s


# -------------------------------------------------------------- plain form

def _act(name, v):
    """The activation and its derivative."""
    if name == "none":
        return v, torch.ones_like(v)
    sig = 1.0 / (1.0 + torch.exp(-v))
    if name == "sigmoid":
        return sig, sig * (1.0 - sig)
    return v * sig, sig * (1.0 + v * (1.0 - sig))


def _extended(s, W):
    """x with the W - 1 rows that enter each sequence laid before its rows, the place there of each of x's
    rows, and the places of each sequence's first and last W - 1 rows."""
    cu, x = s["cu"].long(), s["x"].float()
    T, N = x.shape[0], cu.shape[0] - 1
    dev = x.device
    seq = torch.repeat_interleave(torch.arange(N, device=dev), cu[1:] - cu[:-1])
    at = torch.arange(T, device=dev) + (seq + 1) * (W - 1)
    taps, ids = torch.arange(W - 1, device=dev), torch.arange(N, device=dev)
    head = (cu[:-1] + ids * (W - 1))[:, None] + taps
    tail = (cu[1:] + ids * (W - 1))[:, None] + taps
    ext = torch.zeros(T + N * (W - 1), x.shape[1], device=dev)
    ext[at] = x
    if s["s0"] is not None:
        ext[head] = s["s0"].float()
    return ext, at, head, tail


def _plain_conv(s):
    case, W = s["case"], s["case"]["W"]
    ext, at, head, tail = _extended(s, W)
    v = torch.zeros_like(ext[at]) if s["b"] is None else s["b"].expand(at.shape[0], -1).clone()
    for j in range(W):
        v += s["w"][:, j] * ext[at - (W - 1) + j]
    y, slope = _act(case["act"], v)
    dt = s["x"].dtype
    fs = ext[tail].to(dt)
    if case["op"] == "conv":
        if s["cache"] is not None:
            keep = s["slots"] >= 0
            s["cache"][s["slots"][keep].long()] = fs[keep]
        return [y.to(dt), fs, s["cache"]]
    dv = s["d_y"].float() * slope
    dext = torch.zeros_like(ext)
    dw = torch.empty_like(s["w"])
    for j in range(W):
        rows = at - (W - 1) + j
        dext[rows] += s["w"][:, j] * dv  # (the rows are distinct)
        dw[:, j] = (dv * ext[rows]).sum(0)
    if s["d_final"] is not None:
        dext[tail] += s["d_final"]
    db = dv.sum(0) if s["b"] is not None else None
    return [y.to(dt), fs, dext[at].to(dt), dw, db, dext[head] if s["s0"] is not None else None]


def _plain_conv_decode(s):
    slots, x = s["slots"], s["x"].float()
    live = torch.nonzero(slots >= 0)[:, 0]
    at = slots[live].long()
    window = torch.cat([s["cache"][at].float(), x[live][:, None]], 1)
    v = (window * s["w"].t()).sum(1)
    if s["b"] is not None:
        v = v + s["b"]
    y = torch.zeros_like(s["x"]).index_copy(0, live, _act(s["case"]["act"], v)[0].to(s["x"].dtype))
    s["cache"][at] = window[:, 1:].to(s["cache"].dtype)
    return [y, s["cache"]]


def _recurrence(a, u):
    """h_t = a_t h_{t-1} + u_t over the rows of [T, ...] float32 tensors from h = 0: a loop over the rows of
    all blocks of about sqrt(T) rows at once, a loop over the blocks' ends, and one product that adds what
    enters each block.  A recurrence needs the loops; these are the shortest of this form."""
    T, C = a.shape[0], 1 << max(0, (a.shape[0] - 1).bit_length() // 2)
    B = -(-T // C)
    if B * C > T:
        a, u = (torch.cat([t, t.new_zeros(B * C - T, *t.shape[1:])]) for t in (a, u))
    a, h = a.unflatten(0, (B, C)).clone(), u.unflatten(0, (B, C)).clone()  # products of decays / states
    for c in range(1, C):
        h[:, c] += a[:, c] * h[:, c - 1]
        a[:, c] *= a[:, c - 1]
    enter = torch.zeros_like(h[:, 0])
    for b in range(1, B):
        enter[b] = a[b - 1, -1] * enter[b - 1] + h[b - 1, -1]
    h += a * enter[:, None]
    return h.flatten(0, 1)[:T]


def _softplus(v):
    """log(1 + exp(v)) and its derivative."""
    return torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-v.abs())), 1.0 / (1.0 + torch.exp(-v))


def _per_channel(t, D):
    """[T, G, S] of the groups as [T, D, S] of their channels."""
    return t.float().repeat_interleave(D // t.shape[1], 1)


def _plain_select(s):
    case, D = s["case"], s["case"]["D"]
    u, A, dt = s["u"].float(), s["A"], s["u"].dtype
    delta, slope = _softplus(s["dt"].float() + s["dt_bias"])
    B, C = _per_channel(s["B"], D), _per_channel(s["C"], D)
    a = torch.exp(delta[:, :, None] * A)
    term = (delta * u)[:, :, None] * B
    live = torch.nonzero(s["cu"][1:] > s["cu"][:-1])[:, 0]
    first, last = s["cu"][:-1][live].long(), s["cu"][1:][live].long() - 1
    if s["s0"] is not None:
        term = term.index_add(0, first, a[first] * s["s0"][live])
    reset = a.index_fill(0, first, 0.0)
    h = _recurrence(reset, term)
    fs = s["s0"].clone() if s["s0"] is not None else torch.zeros(s["cu"].shape[0] - 1, *h.shape[1:], device=h.device)
    fs = fs.index_copy(0, live, h[last])
    pre = (h * C).sum(-1) + s["skip"] * u
    f, df = (1.0, 0.0) if s["z"] is None else _act("silu", s["z"].float())
    o = (pre * f).to(dt)
    if case["op"] == "select":
        if s["cache"] is not None:
            keep = s["slots"] >= 0
            s["cache"][s["slots"][keep].long()] = fs[keep]
        return [o, fs, s["cache"]]
    d_o = s["d_o"].float()
    dz = None if s["z"] is None else (d_o * pre * df).to(dt)
    gy = d_o * f
    d = gy[:, :, None] * C
    if s["d_final"] is not None:
        d.index_add_(0, last, s["d_final"][live])
    e = _recurrence(torch.cat([reset[1:], torch.zeros_like(reset[:1])]).flip(0), d.flip(0)).flip(0)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[first] = s["s0"][live] if s["s0"] is not None else 0.0
    carried = e * a * before
    through = (e * B).sum(-1)
    ddelta = (carried * A).sum(-1) + u * through
    groups = lambda t: t.unflatten(1, (case["G"], D // case["G"])).sum(2).to(dt)  # noqa: E731
    ds0 = None
    if s["s0"] is not None:
        ds0 = s["d_final"].clone().index_copy(0, live, a[first] * e[first])
    ddt = ddelta * slope
    return [o, fs, (gy * s["skip"] + delta * through).to(dt), ddt.to(s["dt"].dtype),
            (carried * delta[:, :, None]).sum(0), groups(e * (delta * u)[:, :, None]), groups(gy[:, :, None] * h),
            (gy * u).sum(0), dz, ddt.sum(0), ds0]


def _plain_select_decode(s):
    D, slots = s["case"]["D"], s["slots"]
    live = torch.nonzero(slots >= 0)[:, 0]
    at = slots[live].long()
    u = s["u"][live].float()
    delta = _softplus(s["dt"][live].float() + s["dt_bias"])[0]
    h = torch.exp(delta[:, :, None] * s["A"]) * s["cache"][at] + (delta * u)[:, :, None] * _per_channel(s["B"][live], D)
    s["cache"][at] = h
    o = (h * _per_channel(s["C"][live], D)).sum(-1) + s["skip"] * u
    if s["z"] is not None:
        o = o * _act("silu", s["z"][live].float())[0]
    return [torch.zeros_like(s["u"]).index_copy(0, live, o.to(s["u"].dtype)), s["cache"]]


def _plain_between(s):
    case, x, y = s["case"], s["x"].float(), s["y"].float()
    hat, rstd = y, 1.0
    if case["post"]:
        rstd = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
        hat = y * rstd
    p = hat * s["w_post"]
    f, df = (1.0, 0.0) if s["z"] is None else _act(case["act"], s["z"].float())
    r = x + case["scale"] * (f * p)
    n = None
    if case["pre"]:
        rr = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
        rhat = r * rr
        n = (rhat * s["w_pre"]).to(s["y"].dtype)
    if case["op"] == "between":
        return [r.to(s["x"].dtype), n]
    dt = s["y"].dtype
    dx, dw_pre = s["d_r"].float(), None
    if case["pre"]:
        dn = s["d_n"].float()
        q = dn * s["w_pre"]
        dx = dx + rr * (q - rhat * (q * rhat).mean(-1, keepdim=True))
        dw_pre = (dn * rhat).sum(0)
    d = case["scale"] * dx
    dz = None if s["z"] is None else (d * p * df).to(dt)
    dp = d * f
    q = dp * s["w_post"]
    dy = rstd * (q - hat * (q * hat).mean(-1, keepdim=True)) if case["post"] else q
    return [r.to(s["x"].dtype), n.to(dt) if case["pre"] else None, dx.to(s["x"].dtype), dy.to(dt), dz,
            (dp * hat).sum(0), dw_pre]


# --------------------------------------------------------------------- run

def run(state):
    s = state
    case = s["case"]
    op = case["op"]
    if own:
        from gated_deltaproduct_recurrence_amd import binding
        if op == "conv_decode":
            y = binding.short_conv_decode(s["x"], s["w"], s["cache"], s["slots"], bias=s["b"], activation=case["act"])
            return [y, s["cache"]]
        if op in ("conv", "conv_train"):
            form = {"bias": s["b"], "activation": case["act"], "initial_state": s["s0"]}
            y, fs = binding.short_conv(s["x"], s["w"], s["cu"], output_final_state=True, state_cache=s["cache"],
                                       state_indices=s["slots"], **form)
            if op == "conv":
                return [y, fs, s["cache"]]
            d = binding.short_conv_backward(s["x"], s["w"], s["cu"], s["d_y"], d_final_state=s["d_final"], **form)
            return [y, fs, d["dx"], d["dweight"], d["dbias"], d["d_initial_state"]]
        if op in ("select", "select_train", "select_decode"):
            args = (s["u"], s["dt"], s["A"], s["B"], s["C"])
            form = {"skip": s["skip"], "gate": s["z"], "dt_bias": s["dt_bias"], "dt_softplus": True}
            if op == "select_decode":
                return [binding.selective_scan_decode(*args, s["cache"], s["slots"], **form), s["cache"]]
            form["initial_state"] = s["s0"]
            if op == "select":
                o, fs = binding.selective_scan(*args, s["cu"], output_final_state=True, state_cache=s["cache"],
                                               state_indices=s["slots"], **form)
                return [o, fs, s["cache"]]
            o, fs, points = binding.selective_scan(*args, s["cu"], output_final_state=True, return_checkpoints=True,
                                                   **form)
            d = binding.selective_scan_backward(*args, s["cu"], s["d_o"], d_final_state=s["d_final"],
                                                checkpoints=points, **form)
            return [o, fs, *(d[k] for k in ("du", "ddt", "dA", "dB", "dC", "dskip", "dgate", "ddt_bias",
                                            "d_initial_state"))]
        form = {"post_weight": s["w_post"], "pre_weight": s["w_pre"], "gate": s["z"], "activation": case["act"],
                "post_norm": case["post"], "pre_norm": case["pre"], "residual_scale": case["scale"], "eps": EPS}
        r, n = binding.residual_norm(s["x"], s["y"], **form)
        if op == "between":
            return [r, n]
        d = binding.residual_norm_backward(s["x"], s["y"], s["d_r"], s["d_n"], **form)
        return [r, n, d["dx"], d["dy"], d["dgate"], d["dpost_weight"], d["dpre_weight"]]
    if op in ("conv", "conv_train"):
        return _plain_conv(s)
    if op == "conv_decode":
        return _plain_conv_decode(s)
    if op in ("select", "select_train"):
        return _plain_select(s)
    if op == "select_decode":
        return _plain_select_decode(s)
    return _plain_between(s)


# -------------------------------------------------------------------- work

def _size(dtype):
    return torch.finfo(DTYPES[dtype]).bits // 8


def work(case):
    e, D, op = _size(case["dtype"]), case["D"], case["op"]
    if op == "conv_decode":
        live, W = case["N"] - case["pad"], case["W"]
        # x read and the state read and written for live entries, y written for all
        return {"bytes": D * (live * e * (2 * W - 1) + case["N"] * e + 4 * W), "flops": live * D * (2 * W + 4)}
    if op in ("conv", "conv_train"):
        lens, W = _lens(case), case["W"]
        T, states = sum(lens), len(lens) * (W - 1) * D * e
        params = 4 * D * (W + bool(case["bias"]))
        if op == "conv":
            n = 1 + bool(case["initial"]) + bool(case["slots"])
            return {"bytes": 2 * T * D * e + n * states + params, "flops": T * D * (2 * W + 4)}
        # x and d_y read, y and dx written; the states' gradients are float32
        carried = states + 2 * states * 4 // e if case["initial"] else 0
        return {"bytes": 4 * T * D * e + states + carried + 2 * params, "flops": T * D * (6 * W + 12)}
    if op in ("select", "select_train", "select_decode"):
        S, G, de, gated = case["S"], case["G"], _size(case["dt"]), bool(case["gated"])
        params = 4 * D * (S + 2)
        if op == "select_decode":
            live = case["N"] - case["pad"]
            row = D * (e * (1 + gated) + de) + 2 * G * S * e
            return {"bytes": live * (row + 8 * D * S) + case["N"] * D * e + params, "flops": live * D * (7 * S + 10)}
        lens = _lens(case)
        T, states = sum(lens), len(lens) * D * S * 4
        row = D * (e * (2 + gated) + de) + 2 * G * S * e
        if op == "select":
            n = 1 + bool(case["initial"]) + bool(case["slots"])
            return {"bytes": T * row + n * states + params, "flops": T * D * (7 * S + 10)}
        # u, dt, B, C, d_o (and the gate) read, o and the gradients of the inputs written
        n = 4 if case["initial"] else 1
        return {"bytes": T * (2 * row + D * e) + n * states + 2 * params, "flops": T * D * (23 * S + 30)}
    T, se, gated = case["T"], _size(case["stream"]), bool(case["gated"])
    params = 4 * D * (1 + bool(case["pre"]))
    if op == "between":
        return {"bytes": T * D * (2 * se + e * (1 + gated + bool(case["pre"]))) + params, "flops": T * D * 14}
    # x, y, d_r, d_n (and the gate) read, r, n, dx, dy (and the gate's gradient) written
    return {"bytes": T * D * (4 * se + e * (2 + 2 * gated + 2 * bool(case["pre"]))) + 2 * params, "flops": T * D * 40}


# ------------------------------------------------------------------- exact

def _order(cu):
    """Sequences by falling length: their numbers, lengths and first rows."""
    edges = cu.tolist()
    order = sorted(range(len(edges) - 1), key=lambda i: edges[i] - edges[i + 1])
    return order, [edges[i + 1] - edges[i] for i in order], [edges[i] for i in order]


def _exact_conv(s, case):
    f64, W = torch.float64, case["W"]
    x, w = s["x"].to(f64), s["w"].to(f64)
    edges = s["cu"].tolist()
    N, D = len(edges) - 1, case["D"]
    s0 = torch.zeros(N, W - 1, D, dtype=f64, device=x.device) if s["s0"] is None else s["s0"].to(f64)
    train = case["op"] == "conv_train"
    y, dx = torch.zeros_like(x), torch.zeros_like(x)
    fs, dw, db, ds0 = torch.zeros_like(s0), torch.zeros_like(w), torch.zeros_like(w[:, 0]), torch.zeros_like(s0)
    for i, (lo, hi) in enumerate(zip(edges, edges[1:])):
        n = hi - lo
        rows = torch.cat([s0[i], x[lo:hi]])
        fs[i] = rows[n:]
        v = torch.stack([rows[j:j + n] for j in range(W)], -1).mul(w).sum(-1)
        if s["b"] is not None:
            v += s["b"]
        sg = torch.sigmoid(v)
        y[lo:hi] = {"none": v, "sigmoid": sg, "silu": v * sg}[case["act"]]
        if not train:
            continue
        slope = {"none": torch.ones_like(v), "sigmoid": sg * (1 - sg), "silu": sg + v * sg * (1 - sg)}[case["act"]]
        dv = s["d_y"][lo:hi].to(f64) * slope
        drows = torch.zeros_like(rows)
        if s["d_final"] is not None:
            drows[n:] += s["d_final"][i].to(f64)
        for j in range(W):
            drows[j:j + n] += w[:, j] * dv
            dw[:, j] += (rows[j:j + n] * dv).sum(0)
        db += dv.sum(0)
        ds0[i], dx[lo:hi] = drows[:W - 1], drows[W - 1:]
    if not train:
        cache = None
        if s["cache"] is not None:
            cache = s["cache"].to(f64)
            for i, slot in enumerate(s["slots"].tolist()):
                if slot >= 0:
                    cache[slot] = fs[i]
        return [y, fs, cache]
    return [y, fs, dx, dw, db if s["b"] is not None else None, ds0 if s["s0"] is not None else None]


def _exact_select(s, case):
    f64, D, S, G = torch.float64, case["D"], case["S"], case["G"]
    u, A, skip = s["u"].to(f64), s["A"].to(f64), s["skip"].to(f64)
    v = s["dt"].to(f64) + s["dt_bias"].to(f64)
    delta = torch.nn.functional.softplus(v, threshold=100.0)
    T, N, dev = u.shape[0], s["cu"].shape[0] - 1, u.device
    wide = lambda t: t.to(f64)[:, :, None].expand(-1, G, D // G, S).reshape(-1, D, S)  # noqa: E731
    order, sizes, starts = _order(s["cu"])
    rank = torch.tensor(order, device=dev)
    start = torch.tensor(starts, device=dev)
    h0 = torch.zeros(N, D, S, dtype=f64, device=dev) if s["s0"] is None else s["s0"].to(f64)
    train = case["op"] == "select_train"
    pre = torch.zeros_like(u)
    before = torch.zeros(T, D, S, dtype=f64, device=dev) if train else None
    h, k = h0[rank], N
    for t in range(max(sizes)):
        while k and sizes[k - 1] <= t:
            k -= 1
        rows = start[:k] + t
        if train:
            before[rows] = h[:k]
        h[:k] = (delta[rows, :, None] * A).exp() * h[:k] + (delta[rows] * u[rows])[:, :, None] * wide(s["B"][rows])
        pre[rows] = (h[:k] * wide(s["C"][rows])).sum(-1) + skip * u[rows]
    fs = torch.zeros_like(h)
    fs[rank] = h
    z = None if s["z"] is None else s["z"].to(f64)
    f = torch.ones_like(u) if z is None else z * torch.sigmoid(z)
    o = pre * f
    if not train:
        cache = None
        if s["cache"] is not None:
            cache = s["cache"].to(f64)
            for i, slot in enumerate(s["slots"].tolist()):
                if slot >= 0:
                    cache[slot] = fs[i]
        return [o, fs, cache]
    d_o = s["d_o"].to(f64)
    gy = d_o * f
    e = torch.zeros(N, D, S, dtype=f64, device=dev) if s["d_final"] is None else s["d_final"].to(f64)[rank]
    end = start + torch.tensor(sizes, device=dev) - 1
    du, dd = torch.zeros_like(u), torch.zeros_like(u)
    dA, dB = torch.zeros_like(A), torch.zeros(T, G, S, dtype=f64, device=dev)
    dC, k = torch.zeros_like(dB), N
    for t in range(max(sizes)):
        while k and sizes[k - 1] <= t:
            k -= 1
        rows = end[:k] - t
        dl, ur, g = delta[rows, :, None], u[rows, :, None], gy[rows, :, None]
        a, Br, hb = (dl * A).exp(), wide(s["B"][rows]), before[rows]
        e[:k] += g * wide(s["C"][rows])
        kept = a * hb
        dC[rows] = (g * (kept + dl * ur * Br)).unflatten(1, (G, D // G)).sum(2)
        dB[rows] = (e[:k] * dl * ur).unflatten(1, (G, D // G)).sum(2)
        du[rows] = (e[:k] * Br).sum(-1) * delta[rows] + gy[rows] * skip
        dd[rows] = (e[:k] * (kept * A + ur * Br)).sum(-1)
        dA += (e[:k] * kept * dl).sum(0)
        e[:k] *= a
    ds0 = torch.zeros_like(e)
    ds0[rank] = e
    ddt = dd * torch.sigmoid(v)
    dz = None
    if z is not None:
        sg = torch.sigmoid(z)
        dz = d_o * pre * (sg + z * sg * (1 - sg))
    return [o, fs, du, ddt, dA, dB, dC, (gy * u).sum(0), dz, ddt.sum(0), ds0 if s["s0"] is not None else None]


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    op = case["op"]
    if op in ("conv", "conv_train"):
        return _exact_conv(s, case)
    if op in ("select", "select_train"):
        return _exact_select(s, case)
    if op == "conv_decode":
        x, w, cache = s["x"].to(f64), s["w"].to(f64), s["cache"].to(f64)
        y = torch.zeros_like(x)
        for i, slot in enumerate(s["slots"].tolist()):
            if slot < 0:
                continue
            window = torch.cat([cache[slot], x[i:i + 1]])
            v = (window.t() * w).sum(1) + (0 if s["b"] is None else s["b"])
            y[i] = {"none": v, "sigmoid": torch.sigmoid(v), "silu": v * torch.sigmoid(v)}[case["act"]]
            cache[slot] = window[1:]
        return [y, cache]
    if op == "select_decode":
        G, S, per = case["G"], case["S"], case["D"] // case["G"]
        cache, A = s["cache"].to(f64), s["A"].to(f64)
        o = torch.zeros(case["N"], case["D"], dtype=f64, device="cuda")
        for i, slot in enumerate(s["slots"].tolist()):
            if slot < 0:
                continue
            u = s["u"][i].to(f64)
            delta = torch.nn.functional.softplus(s["dt"][i].to(f64) + s["dt_bias"].to(f64), threshold=100.0)
            B, C = (s[k][i].to(f64)[:, None].expand(G, per, S).reshape(-1, S) for k in "BC")
            cache[slot] = (delta[:, None] * A).exp() * cache[slot] + (delta * u)[:, None] * B
            o[i] = (cache[slot] * C).sum(1) + s["skip"].to(f64) * u
            if s["z"] is not None:
                z = s["z"][i].to(f64)
                o[i] *= z * torch.sigmoid(z)
        return [o, cache]
    x, y, D, c = s["x"].to(f64), s["y"].to(f64), case["D"], float(case["scale"])
    wp = s["w_post"].to(f64)
    ry = ((y ** 2).sum(-1, keepdim=True) / D + EPS) ** -0.5 if case["post"] else torch.ones_like(y[:, :1])
    f, df = torch.ones_like(y), torch.zeros_like(y)
    if s["z"] is not None:
        z = s["z"].to(f64)
        sg = torch.sigmoid(z)
        f = {"none": z, "sigmoid": sg, "silu": z * sg}[case["act"]]
        df = {"none": torch.ones_like(z), "sigmoid": sg * (1 - sg), "silu": sg + z * sg * (1 - sg)}[case["act"]]
    r = x + c * f * (y * ry) * wp
    rr = ((r ** 2).sum(-1, keepdim=True) / D + EPS) ** -0.5
    n = r * rr * s["w_pre"].to(f64) if case["pre"] else None
    if op == "between":
        return [r, n]
    dr, dw_pre = s["d_r"].to(f64), None
    if case["pre"]:
        dn = s["d_n"].to(f64)
        dw_pre = (dn * r * rr).sum(0)
        g = dn * s["w_pre"].to(f64)
        dr = dr + rr * g - r * rr ** 3 * ((g * r).sum(-1, keepdim=True) / D)
    g = c * dr * f * wp
    dy = ry * g - y * ry ** 3 * ((g * y).sum(-1, keepdim=True) / D) if case["post"] else g
    return [r, n, dr, dy, c * dr * (y * ry) * wp * df if s["z"] is not None else None,
            (c * dr * f * (y * ry)).sum(0), dw_pre]
