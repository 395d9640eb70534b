"""ctypes binding of libgdp.so (include/gdp.h), same names as the C ABI.

Argument marshalling only: torch supplies device memory and the current
stream; every step of the computation runs in the library's HIP kernels.  If
the library is missing this module raises on import -- there is no fallback.
The entries of the layers (gated scan, group norm, short convolution,
selective scan, residual norm) also need the extension _records.so, built for
this Python and torch; without it they raise when called, and the others work.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# GDP_LIBRARY names another build of the library (the host-sanitized check
# build of the CPU sanitizer run); by default the in-tree libgdp.so
LIB_PATH = os.environ.get("GDP_LIBRARY") or os.path.join(_HERE, "libgdp.so")

GDP_F32, GDP_BF16, GDP_I32, GDP_I64, GDP_F16 = 0, 1, 2, 3, 4
GDP_OK, GDP_EINVAL, GDP_EUNSUPPORTED, GDP_EALIAS, GDP_EWORKSPACE, GDP_EHIP = 0, -1, -2, -3, -4, -5
GDP_DBG_CU, GDP_DBG_SLOT, GDP_DBG_DUP = 1, 2, 4
GDP_SCAN_CHECKPOINT_ROWS = 64
GDP_SELECT_CHECKPOINT_ROWS = 16
ACTIVATIONS = {None: 0, "none": 0, "silu": 1, "sigmoid": 2}  # gdp_activation
STATUS_NAMES = {GDP_EINVAL: "GDP_EINVAL", GDP_EUNSUPPORTED: "GDP_EUNSUPPORTED", GDP_EALIAS: "GDP_EALIAS",
                GDP_EWORKSPACE: "GDP_EWORKSPACE", GDP_EHIP: "GDP_EHIP"}

EXPORTED = ("gdp_descriptor_capacity", "gdp_build_descriptors", "gdp_workspace_bytes",
            "gdp_chunk_prefill", "gdp_recurrent_decode", "gdp_fi_workspace_bytes",
            "gdp_chunk_gated_delta_product", "gdp_backward_workspace_bytes", "gdp_chunk_prefill_backward",
            "gdp_debug_status", "gdp_last_error", "gdp_version", "gdp_chunk_prefill_noalloc",
            "gdp_gated_scan_workspace_bytes", "gdp_gated_scan", "gdp_gated_scan_decode",
            "gdp_gated_scan_backward_workspace_bytes", "gdp_gated_scan_backward", "gdp_group_norm",
            "gdp_group_norm_backward_workspace_bytes", "gdp_group_norm_backward",
            "gdp_short_conv", "gdp_short_conv_decode", "gdp_short_conv_backward_workspace_bytes",
            "gdp_short_conv_backward", "gdp_selective_scan_workspace_bytes", "gdp_selective_scan",
            "gdp_selective_scan_decode", "gdp_selective_scan_backward_workspace_bytes",
            "gdp_selective_scan_backward", "gdp_residual_norm", "gdp_residual_norm_backward_workspace_bytes",
            "gdp_residual_norm_backward")


class gdp_tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


class gdp_descriptors(ctypes.Structure):
    _fields_ = [("chunk_indices", ctypes.c_void_p), ("chunk_indices_dp", ctypes.c_void_p),
                ("chunk_offsets", ctypes.c_void_p), ("chunk_offsets_dp", ctypes.c_void_p),
                ("nt_cap", ctypes.c_int64), ("ntdp_cap", ctypes.c_int64)]


class GdpError(RuntimeError):
    def __init__(self, code, message):
        super().__init__(f"{STATUS_NAMES.get(code, code)}: {message}")
        self.code = code


def _load(path=LIB_PATH):
    if not os.path.exists(path):
        raise ImportError(f"{path} is not built; run __graft_entry__.build() "
                          "(gated_deltaproduct_recurrence_amd/build.py)")
    lib = ctypes.CDLL(path)
    T = ctypes.POINTER(gdp_tensor)
    D = ctypes.POINTER(gdp_descriptors)
    lib.gdp_descriptor_capacity.restype = ctypes.c_int
    lib.gdp_descriptor_capacity.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                            ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int64)]
    lib.gdp_build_descriptors.restype = ctypes.c_int
    lib.gdp_build_descriptors.argtypes = [T, ctypes.c_int32, ctypes.c_int64, D, ctypes.c_void_p]
    lib.gdp_workspace_bytes.restype = ctypes.c_size_t
    lib.gdp_workspace_bytes.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                        ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]
    lib.gdp_chunk_prefill.restype = ctypes.c_int
    lib.gdp_chunk_prefill.argtypes = [T, T, T, T, T, ctypes.c_int32, T, ctypes.c_float, T, ctypes.c_int32,
                                      ctypes.c_int32, T, T, ctypes.c_int32, T, T, T, D, ctypes.c_void_p,
                                      ctypes.c_size_t, ctypes.c_void_p]
    lib.gdp_chunk_prefill_noalloc.restype = ctypes.c_int
    lib.gdp_chunk_prefill_noalloc.argtypes = [T, T, T, T, T, ctypes.c_int32, T, ctypes.c_float, T, ctypes.c_int32,
                                              ctypes.c_int32, T, T, ctypes.c_int32, T, T, T, D, ctypes.c_void_p]
    lib.gdp_recurrent_decode.restype = ctypes.c_int
    lib.gdp_recurrent_decode.argtypes = [T, T, T, T, T, ctypes.c_int32, ctypes.c_float, ctypes.c_int32, T, T, T,
                                         ctypes.c_void_p]
    lib.gdp_fi_workspace_bytes.restype = ctypes.c_size_t
    lib.gdp_fi_workspace_bytes.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                           ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                           ctypes.c_int32]
    lib.gdp_chunk_gated_delta_product.restype = ctypes.c_int
    lib.gdp_chunk_gated_delta_product.argtypes = [T, T, T, T, T, ctypes.c_int32, ctypes.c_float, T,
                                                  ctypes.c_int32, T, ctypes.c_int32, T, T, ctypes.c_void_p,
                                                  ctypes.c_size_t, ctypes.c_void_p]
    lib.gdp_backward_workspace_bytes.restype = ctypes.c_size_t
    lib.gdp_backward_workspace_bytes.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                                 ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]
    lib.gdp_chunk_prefill_backward.restype = ctypes.c_int
    lib.gdp_chunk_prefill_backward.argtypes = [T, T, T, T, T, ctypes.c_int32, T, ctypes.c_float, T, ctypes.c_int32,
                                               T, T, T, T, T, T, T, T, ctypes.c_void_p, ctypes.c_size_t,
                                               ctypes.c_void_p]
    lib.gdp_debug_status.restype = ctypes.c_int
    lib.gdp_debug_status.argtypes = [ctypes.POINTER(ctypes.c_uint32), ctypes.c_int32, ctypes.c_void_p]
    # the layers' tensors cross as addresses of gdp_tensor records (_records)
    P, i32, i64, size = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    for name in ("gdp_gated_scan_workspace_bytes", "gdp_gated_scan_backward_workspace_bytes",
                 "gdp_group_norm_backward_workspace_bytes"):
        getattr(lib, name).restype = size
        getattr(lib, name).argtypes = [i64, i64, i64]
    lib.gdp_gated_scan.restype = ctypes.c_int
    lib.gdp_gated_scan.argtypes = [P, P, P, i32, P, i32, P, P, i32, P, P, P, P, size, P]
    lib.gdp_gated_scan_decode.restype = ctypes.c_int
    lib.gdp_gated_scan_decode.argtypes = [P, P, i32, P, P, P, P]
    lib.gdp_gated_scan_backward.restype = ctypes.c_int
    lib.gdp_gated_scan_backward.argtypes = [P, P, P, i32, P, P, P, P, P, P, P, P, size, P]
    lib.gdp_group_norm.restype = ctypes.c_int
    lib.gdp_group_norm.argtypes = [P, P, P, P, i32, i32, ctypes.c_float, P, P]
    lib.gdp_group_norm_backward.restype = ctypes.c_int
    lib.gdp_group_norm_backward.argtypes = [P, P, P, P, i32, i32, ctypes.c_float, P, P, P, P, P, P, size, P]
    lib.gdp_short_conv.restype = ctypes.c_int
    lib.gdp_short_conv.argtypes = [P, P, P, i32, P, P, i32, P, P, P, P, P]
    lib.gdp_short_conv_decode.restype = ctypes.c_int
    lib.gdp_short_conv_decode.argtypes = [P, P, P, i32, P, P, P, P]
    lib.gdp_short_conv_backward_workspace_bytes.restype = size
    lib.gdp_short_conv_backward_workspace_bytes.argtypes = [i64, i64, i64, i64]
    lib.gdp_short_conv_backward.restype = ctypes.c_int
    lib.gdp_short_conv_backward.argtypes = [P, P, P, i32, P, P, P, P, P, P, P, P, P, size, P]
    lib.gdp_selective_scan_workspace_bytes.restype = size
    lib.gdp_selective_scan_workspace_bytes.argtypes = [i64, i64, i64, i64, i64]
    lib.gdp_selective_scan.restype = ctypes.c_int
    lib.gdp_selective_scan.argtypes = [P, P, P, P, P, P, P, P, i32, P, P, i32, P, P, i32, P, P, P, P, size, P]
    lib.gdp_selective_scan_decode.restype = ctypes.c_int
    lib.gdp_selective_scan_decode.argtypes = [P, P, P, P, P, P, P, P, i32, P, P, P, P]
    lib.gdp_selective_scan_backward_workspace_bytes.restype = size
    lib.gdp_selective_scan_backward_workspace_bytes.argtypes = [i64, i64, i64, i64, i64, i32]
    lib.gdp_selective_scan_backward.restype = ctypes.c_int
    lib.gdp_selective_scan_backward.argtypes = [P, P, P, P, P, P, P, P, i32, *[P] * 15, size, P]
    lib.gdp_residual_norm.restype = ctypes.c_int
    lib.gdp_residual_norm.argtypes = [P, P, P, P, P, i32, i32, i32, ctypes.c_float, ctypes.c_float, P, P, P]
    lib.gdp_residual_norm_backward_workspace_bytes.restype = size
    lib.gdp_residual_norm_backward_workspace_bytes.argtypes = [i64, i64]
    lib.gdp_residual_norm_backward.restype = ctypes.c_int
    lib.gdp_residual_norm_backward.argtypes = [P, P, P, P, P, i32, i32, i32, ctypes.c_float, ctypes.c_float,
                                               *[P] * 8, size, P]
    lib.gdp_last_error.restype = ctypes.c_char_p
    lib.gdp_last_error.argtypes = []
    lib.gdp_version.restype = ctypes.c_char_p
    lib.gdp_version.argtypes = []
    return lib


LIB = _load()


def _load_records():
    """records() of the extension; where that is missing or built for something else, one that says so."""
    try:
        from . import _records as ext  # (after torch, whose libraries it needs)
        if ext.record_bytes != ctypes.sizeof(gdp_tensor):
            raise ImportError(f"it fills records of {ext.record_bytes} bytes, gdp_tensor has {ctypes.sizeof(gdp_tensor)}")
        return ext.records
    except (ImportError, AttributeError) as e:
        why = str(e)

    def records(*_):
        raise ImportError(f"the binding's extension is not built for this library, Python and torch ({why}); run "
                          "__graft_entry__.build() (gated_deltaproduct_recurrence_amd/build.py)")
    return records


_records = _load_records()

_DT = {torch.float32: GDP_F32, torch.bfloat16: GDP_BF16, torch.int32: GDP_I32, torch.int64: GDP_I64,
       torch.float16: GDP_F16}


def as_gdp_tensor(t):
    """gdp_tensor view of a torch tensor (None -> absent)."""
    g = gdp_tensor()
    if t is None:
        return g
    if t.dim() > 4:
        raise ValueError("at most 4 dims")
    if t.dtype not in _DT:
        raise ValueError(f"unsupported dtype {t.dtype}")
    g.data = t.data_ptr() if t.numel() > 0 else None
    g.dtype = _DT[t.dtype]
    g.ndim = t.dim()
    for d in range(t.dim()):
        g.shape[d] = t.shape[d]
        g.stride[d] = t.stride(d)
    if t.numel() == 0:
        # an empty tensor is still "present"; give it a non-null dummy address
        g.data = 16
    return g


def _check(rc):
    if rc != GDP_OK:
        raise GdpError(rc, LIB.gdp_last_error().decode())


def _stream(device):
    return torch.cuda.current_stream(device).cuda_stream


# the current stream's handle and the current device without the Python objects around them (2 us less
# a call), where torch has them
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _empty(like, shape=None, dtype=None):
    """A new contiguous tensor on `like`'s device, by default of its shape and dtype."""
    if shape is None:
        return torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format)
    return like.new_empty(shape, dtype=dtype)


def _workspace(like, nbytes):
    return like.new_empty(nbytes, dtype=torch.uint8) if nbytes else None


# ---------------------------------------------------------------- C ABI names

def gdp_version():
    return LIB.gdp_version().decode()


def gdp_last_error():
    return LIB.gdp_last_error().decode()


def gdp_debug_status(clear=True, device=None):
    """The current device's debug-validation word (GDP_DBG_* bits) after the work
    queued on the current stream; cleared afterwards when `clear`.  The checks run
    only with GDP_DEBUG_VALIDATE=1 in the environment."""
    word = ctypes.c_uint32(0)
    _check(LIB.gdp_debug_status(ctypes.byref(word), 1 if clear else 0, _stream(device)))
    return int(word.value)


def gdp_descriptor_capacity(T, N, num_householder):
    a, b = ctypes.c_int64(), ctypes.c_int64()
    _check(LIB.gdp_descriptor_capacity(T, N, num_householder, ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def gdp_workspace_bytes(T, N, num_householder, Hqk, Hv, K, V, dtype=torch.bfloat16):
    return int(LIB.gdp_workspace_bytes(T, N, num_householder, Hqk, Hv, K, V, _DT[dtype]))


def gdp_build_descriptors(cu_seqlens, num_householder, T, nt_cap=None, ntdp_cap=None, out=None):
    """Device-built descriptors of both chunkings (int32 tensors), padded to capacity.

    ``out``: a dict of caller-allocated buffers (as this function returns) to
    build into, with the capacities their row counts give; nothing is then
    allocated, so the call can be captured in a graph."""
    N = cu_seqlens.shape[0] - 1
    dev = cu_seqlens.device
    if out is None:
        ct, cd = gdp_descriptor_capacity(T, N, num_householder)
        nt_cap = ct if nt_cap is None else nt_cap
        ntdp_cap = cd if ntdp_cap is None else ntdp_cap
        out = {"chunk_indices": torch.empty((max(nt_cap, 1), 2), dtype=torch.int32, device=dev),
               "chunk_indices_dp": torch.empty((max(ntdp_cap, 1), 2), dtype=torch.int32, device=dev),
               "chunk_offsets": torch.empty(N + 1, dtype=torch.int32, device=dev),
               "chunk_offsets_dp": torch.empty(N + 1, dtype=torch.int32, device=dev)}
    else:
        nt_cap, ntdp_cap = out["chunk_indices"].shape[0], out["chunk_indices_dp"].shape[0]
    d = _descs(out, nt_cap, ntdp_cap)
    cu = as_gdp_tensor(cu_seqlens)
    _check(LIB.gdp_build_descriptors(ctypes.byref(cu), num_householder, T, ctypes.byref(d), _stream(dev)))
    out["chunk_indices"] = out["chunk_indices"][:nt_cap]
    out["chunk_indices_dp"] = out["chunk_indices_dp"][:ntdp_cap]
    return out


def _descs(dct, nt_cap, ntdp_cap):
    d = gdp_descriptors()
    d.chunk_indices = dct["chunk_indices"].data_ptr()
    d.chunk_indices_dp = dct["chunk_indices_dp"].data_ptr()
    d.chunk_offsets = dct["chunk_offsets"].data_ptr()
    d.chunk_offsets_dp = dct["chunk_offsets_dp"].data_ptr()
    d.nt_cap = nt_cap
    d.ntdp_cap = ntdp_cap
    return d


def gdp_chunk_prefill(q, k, v, g_log, beta, num_householder, cu_seqlens, scale=0.0, initial_state=None,
                      output_final_state=False, use_qk_l2norm=False, state_cache=None, state_indices=None,
                      return_chunk_states=False, o=None, final_state=None, chunk_states=None,
                      descriptors=None, workspace=None, stream=None):
    """Direct call of the C entry point with caller-allocated outputs (all torch tensors).

    ``descriptors`` is a dict as returned by gdp_build_descriptors or None;
    ``workspace`` is a uint8 device tensor of at least gdp_workspace_bytes(...)
    bytes."""
    args = [as_gdp_tensor(x) for x in (q, k, v, g_log, beta)]
    cu = as_gdp_tensor(cu_seqlens)
    s0 = as_gdp_tensor(initial_state)
    cache = as_gdp_tensor(state_cache)
    slots = as_gdp_tensor(state_indices)
    ot, ft, ct = as_gdp_tensor(o), as_gdp_tensor(final_state), as_gdp_tensor(chunk_states)
    dptr = None
    if descriptors is not None:
        d = _descs(descriptors, descriptors["chunk_indices"].shape[0], descriptors["chunk_indices_dp"].shape[0])
        dptr = ctypes.byref(d)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = _stream(q.device) if stream is None else stream
    rc = LIB.gdp_chunk_prefill(*[ctypes.byref(a) for a in args], int(num_householder), ctypes.byref(cu),
                               float(scale or 0.0), ctypes.byref(s0), int(bool(output_final_state)),
                               int(bool(use_qk_l2norm)), ctypes.byref(cache), ctypes.byref(slots),
                               int(bool(return_chunk_states)), ctypes.byref(ot), ctypes.byref(ft),
                               ctypes.byref(ct), dptr, ws_ptr, ws_bytes, st)
    _check(rc)


def gdp_chunk_prefill_noalloc(q, k, v, g_log, beta, num_householder, cu_seqlens, scale=0.0, initial_state=None,
                              output_final_state=False, use_qk_l2norm=False, state_cache=None, state_indices=None,
                              return_chunk_states=False, o=None, final_state=None, chunk_states=None,
                              descriptors=None, stream=None):
    """Direct call of the C entry point that takes no workspace (its scratch is
    the library's static per-GPU array); outputs are caller-allocated."""
    args = [as_gdp_tensor(x) for x in (q, k, v, g_log, beta)]
    cu = as_gdp_tensor(cu_seqlens)
    s0 = as_gdp_tensor(initial_state)
    cache = as_gdp_tensor(state_cache)
    slots = as_gdp_tensor(state_indices)
    ot, ft, ct = as_gdp_tensor(o), as_gdp_tensor(final_state), as_gdp_tensor(chunk_states)
    dptr = None
    if descriptors is not None:
        d = _descs(descriptors, descriptors["chunk_indices"].shape[0], descriptors["chunk_indices_dp"].shape[0])
        dptr = ctypes.byref(d)
    st = _stream(q.device) if stream is None else stream
    rc = LIB.gdp_chunk_prefill_noalloc(*[ctypes.byref(a) for a in args], int(num_householder), ctypes.byref(cu),
                                       float(scale or 0.0), ctypes.byref(s0), int(bool(output_final_state)),
                                       int(bool(use_qk_l2norm)), ctypes.byref(cache), ctypes.byref(slots),
                                       int(bool(return_chunk_states)), ctypes.byref(ot), ctypes.byref(ft),
                                       ctypes.byref(ct), dptr, st)
    _check(rc)


def gdp_recurrent_decode(q, k, v, g_log, beta, num_householder, scale, use_qk_l2norm, state_cache,
                         state_indices, o, stream=None):
    """Direct call of the C entry point; o is caller-allocated, state_cache is updated in place."""
    args = [as_gdp_tensor(x) for x in (q, k, v, g_log, beta)]
    cache, slots, ot = as_gdp_tensor(state_cache), as_gdp_tensor(state_indices), as_gdp_tensor(o)
    st = _stream(q.device) if stream is None else stream
    _check(LIB.gdp_recurrent_decode(*[ctypes.byref(a) for a in args], int(num_householder), float(scale or 0.0),
                                    int(bool(use_qk_l2norm)), ctypes.byref(cache), ctypes.byref(slots),
                                    ctypes.byref(ot), st))


def gdp_fi_workspace_bytes(T, N, num_householder, Hq, Hv, head_size, dtype=torch.bfloat16,
                           with_initial_state=False, output_final_state=False):
    return int(LIB.gdp_fi_workspace_bytes(T, N, num_householder, Hq, Hv, head_size, _DT[dtype],
                                          int(bool(with_initial_state)), int(bool(output_final_state))))


def gdp_chunk_gated_delta_product(q, k, v, g, beta, num_householder, scale, initial_state, output_final_state,
                                  cu_seqlens, use_qk_l2norm_in_kernel, output, output_state, workspace,
                                  stream=None):
    """Direct call of the FlashInfer-convention C entry point (caller-allocated
    output, output_state and workspace)."""
    ts = [as_gdp_tensor(x) for x in (q, k, v, g, beta)]
    s0, cu = as_gdp_tensor(initial_state), as_gdp_tensor(cu_seqlens)
    ot, st_out = as_gdp_tensor(output), as_gdp_tensor(output_state)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = _stream(q.device) if stream is None else stream
    _check(LIB.gdp_chunk_gated_delta_product(*[ctypes.byref(a) for a in ts], int(num_householder),
                                             float(scale or 0.0), ctypes.byref(s0), int(bool(output_final_state)),
                                             ctypes.byref(cu), int(bool(use_qk_l2norm_in_kernel)),
                                             ctypes.byref(ot), ctypes.byref(st_out), ws_ptr, ws_bytes, st))


def gdp_backward_workspace_bytes(T, N, num_householder, Hqk, Hv, K, V, dtype=torch.bfloat16):
    return int(LIB.gdp_backward_workspace_bytes(T, N, num_householder, Hqk, Hv, K, V, _DT[dtype]))


def gdp_chunk_prefill_backward(q, k, v, g_log, beta, num_householder, cu_seqlens, scale, initial_state,
                               use_qk_l2norm, d_o, d_final_state, dq, dk, dv, dg_log, dbeta, d_initial_state,
                               workspace, stream=None):
    """Direct call of the backward C entry point (caller-allocated gradients and workspace)."""
    ts = [as_gdp_tensor(x) for x in (q, k, v, g_log, beta)]
    cu, s0 = as_gdp_tensor(cu_seqlens), as_gdp_tensor(initial_state)
    dts = [as_gdp_tensor(x) for x in (d_o, d_final_state, dq, dk, dv, dg_log, dbeta, d_initial_state)]
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = _stream(q.device) if stream is None else stream
    _check(LIB.gdp_chunk_prefill_backward(*[ctypes.byref(a) for a in ts], int(num_householder), ctypes.byref(cu),
                                          float(scale or 0.0), ctypes.byref(s0), int(bool(use_qk_l2norm)),
                                          *[ctypes.byref(a) for a in dts], ws_ptr, ws_bytes, st))


def gdp_gated_scan_workspace_bytes(T, N, D):
    return int(LIB.gdp_gated_scan_workspace_bytes(T, N, D))


def gdp_gated_scan_backward_workspace_bytes(T, N, D):
    return int(LIB.gdp_gated_scan_backward_workspace_bytes(T, N, D))


def gdp_group_norm_backward_workspace_bytes(T, G, V):
    return int(LIB.gdp_group_norm_backward_workspace_bytes(T, G, V))


def _call(index, stream, entry, *args):
    """Calls a C entry point on the stream to launch on (None: the current one of the GPU `index`), with
    that GPU as the current device.  The tensors were checked by _records to be there."""
    if index < 0:
        raise ValueError("expected tensors on a GPU, got tensors on the host")
    if index == _current_device():
        rc = entry(*args, _raw_stream(index) if stream is None else stream)
    else:
        with torch.cuda.device(index):
            rc = entry(*args, _raw_stream(index) if stream is None else stream)
    if rc:
        _check(rc)


def _workspace_args(workspace, index):
    if workspace is None:
        return None, 0
    if workspace.get_device() != index:
        raise ValueError(f"expected a workspace on cuda:{index}, got one on {workspace.device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def gdp_gated_scan(x, g_log, cu_seqlens, complement_input, initial_state, output_final_state, state_cache,
                   state_indices, return_checkpoints, o, final_state, checkpoints, workspace, stream=None):
    """Direct call of the C entry point (caller-allocated outputs and workspace)."""
    dev = x.get_device()
    r = _records(dev, x, g_log, cu_seqlens, initial_state, state_cache, state_indices, o, final_state, checkpoints)
    _call(dev, stream, LIB.gdp_gated_scan, r[0], r[1], r[2], bool(complement_input), r[3], bool(output_final_state),
          r[4], r[5], bool(return_checkpoints), r[6], r[7], r[8], *_workspace_args(workspace, dev))


def gdp_gated_scan_decode(x, g_log, complement_input, state_cache, state_indices, o, stream=None):
    """Direct call of the C entry point; o is caller-allocated, state_cache is updated in place."""
    dev = x.get_device()
    r = _records(dev, x, g_log, state_cache, state_indices, o)
    _call(dev, stream, LIB.gdp_gated_scan_decode, r[0], r[1], bool(complement_input), r[2], r[3], r[4])


def gdp_gated_scan_backward(x, g_log, cu_seqlens, complement_input, initial_state, checkpoints, d_o, d_final_state,
                            dx, dg_log, d_initial_state, workspace, stream=None):
    """Direct call of the C entry point (caller-allocated gradients and workspace)."""
    dev = x.get_device()
    r = _records(dev, x, g_log, cu_seqlens, initial_state, checkpoints, d_o, d_final_state, dx, dg_log,
                 d_initial_state)
    _call(dev, stream, LIB.gdp_gated_scan_backward, r[0], r[1], r[2], bool(complement_input), *r[3:10],
          *_workspace_args(workspace, dev))


def gdp_group_norm(x, weight, bias, gate, activation, subtract_mean, eps, y, stream=None):
    """Direct call of the C entry point; `activation` is a key of ACTIVATIONS, y is caller-allocated."""
    dev = x.get_device()
    r = _records(dev, x, weight, bias, gate, y)
    _call(dev, stream, LIB.gdp_group_norm, r[0], r[1], r[2], r[3], _activation(activation), bool(subtract_mean),
          float(eps), r[4])


def gdp_group_norm_backward(x, weight, bias, gate, activation, subtract_mean, eps, d_y, dx, dweight, dbias, dgate,
                            workspace, stream=None):
    """Direct call of the C entry point (caller-allocated gradients and workspace)."""
    dev = x.get_device()
    r = _records(dev, x, weight, bias, gate, d_y, dx, dweight, dbias, dgate)
    _call(dev, stream, LIB.gdp_group_norm_backward, r[0], r[1], r[2], r[3], _activation(activation),
          bool(subtract_mean), float(eps), *r[4:9], *_workspace_args(workspace, dev))


def gdp_short_conv(x, weight, bias, activation, cu_seqlens, initial_state, output_final_state, state_cache,
                   state_indices, y, final_state, stream=None):
    """Direct call of the C entry point (caller-allocated outputs); `activation` is a key of ACTIVATIONS."""
    dev = x.get_device()
    r = _records(dev, x, weight, bias, cu_seqlens, initial_state, state_cache, state_indices, y, final_state)
    _call(dev, stream, LIB.gdp_short_conv, r[0], r[1], r[2], _activation(activation), r[3], r[4],
          bool(output_final_state), r[5], r[6], r[7], r[8])


def gdp_short_conv_decode(x, weight, bias, activation, state_cache, state_indices, y, stream=None):
    """Direct call of the C entry point; y is caller-allocated, state_cache is updated in place."""
    dev = x.get_device()
    r = _records(dev, x, weight, bias, state_cache, state_indices, y)
    _call(dev, stream, LIB.gdp_short_conv_decode, r[0], r[1], r[2], _activation(activation), r[3], r[4], r[5])


def gdp_short_conv_backward_workspace_bytes(T, N, D, W):
    return int(LIB.gdp_short_conv_backward_workspace_bytes(T, N, D, W))


def gdp_short_conv_backward(x, weight, bias, activation, cu_seqlens, initial_state, d_y, d_final_state, dx, dweight,
                            dbias, d_initial_state, workspace, stream=None):
    """Direct call of the C entry point (caller-allocated gradients and workspace)."""
    dev = x.get_device()
    r = _records(dev, x, weight, bias, cu_seqlens, initial_state, d_y, d_final_state, dx, dweight, dbias,
                 d_initial_state)
    _call(dev, stream, LIB.gdp_short_conv_backward, r[0], r[1], r[2], _activation(activation), *r[3:11],
          *_workspace_args(workspace, dev))


def gdp_selective_scan_workspace_bytes(T, N, D, G, S):
    return int(LIB.gdp_selective_scan_workspace_bytes(T, N, D, G, S))


def gdp_selective_scan(u, dt, A, B, C, skip, gate, dt_bias, dt_softplus, cu_seqlens, initial_state,
                       output_final_state, state_cache, state_indices, return_checkpoints, o, final_state,
                       checkpoints, workspace, stream=None):
    """Direct call of the C entry point (caller-allocated outputs and workspace)."""
    dev = u.get_device()
    r = _records(dev, u, dt, A, B, C, skip, gate, dt_bias, cu_seqlens, initial_state, state_cache, state_indices, o,
                 final_state, checkpoints)
    _call(dev, stream, LIB.gdp_selective_scan, *r[:8], bool(dt_softplus), r[8], r[9], bool(output_final_state),
          r[10], r[11], bool(return_checkpoints), r[12], r[13], r[14], *_workspace_args(workspace, dev))


def gdp_selective_scan_decode(u, dt, A, B, C, skip, gate, dt_bias, dt_softplus, state_cache, state_indices, o,
                              stream=None):
    """Direct call of the C entry point; o is caller-allocated, state_cache is updated in place."""
    dev = u.get_device()
    r = _records(dev, u, dt, A, B, C, skip, gate, dt_bias, state_cache, state_indices, o)
    _call(dev, stream, LIB.gdp_selective_scan_decode, *r[:8], bool(dt_softplus), r[8], r[9], r[10])


def gdp_selective_scan_backward_workspace_bytes(T, N, D, G, S, with_checkpoints):
    return int(LIB.gdp_selective_scan_backward_workspace_bytes(T, N, D, G, S, int(bool(with_checkpoints))))


def gdp_selective_scan_backward(u, dt, A, B, C, skip, gate, dt_bias, dt_softplus, cu_seqlens, initial_state,
                                checkpoints, d_o, d_final_state, du, ddt, dA, dB, dC, dskip, dgate, ddt_bias,
                                d_initial_state, workspace, stream=None):
    """Direct call of the C entry point (caller-allocated gradients and workspace)."""
    dev = u.get_device()
    r = _records(dev, u, dt, A, B, C, skip, gate, dt_bias, cu_seqlens, initial_state, checkpoints, d_o,
                 d_final_state, du, ddt, dA, dB, dC, dskip, dgate, ddt_bias, d_initial_state)
    _call(dev, stream, LIB.gdp_selective_scan_backward, *r[:8], bool(dt_softplus), *r[8:22],
          *_workspace_args(workspace, dev))


def gdp_residual_norm(x, y, post_weight, pre_weight, gate, activation, post_norm, pre_norm, residual_scale, eps, r, n,
                      stream=None):
    """Direct call of the C entry point (caller-allocated outputs; r may be x, updated in place)."""
    dev = y.get_device()
    t = _records(dev, x, y, post_weight, pre_weight, gate, r, n)
    _call(dev, stream, LIB.gdp_residual_norm, *t[:5], _activation(activation), bool(post_norm), bool(pre_norm),
          float(residual_scale), float(eps), t[5], t[6])


def gdp_residual_norm_backward_workspace_bytes(T, D):
    return int(LIB.gdp_residual_norm_backward_workspace_bytes(T, D))


def gdp_residual_norm_backward(x, y, post_weight, pre_weight, gate, activation, post_norm, pre_norm, residual_scale,
                               eps, d_r, d_n, dx, dy, dpost_weight, dpre_weight, dgate, workspace, stream=None):
    """Direct call of the C entry point (caller-allocated gradients and workspace)."""
    dev = y.get_device()
    t = _records(dev, x, y, post_weight, pre_weight, gate, d_r, d_n, dx, dy, dpost_weight, dpre_weight, dgate)
    _call(dev, stream, LIB.gdp_residual_norm_backward, *t[:5], _activation(activation), bool(post_norm),
          bool(pre_norm), float(residual_scale), float(eps), *t[5:12], *_workspace_args(workspace, dev))


def _activation(name):
    if name not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(k for k in ACTIVATIONS if k)} or None, got {name!r}")
    return ACTIVATIONS[name]


# ---------------------------------------------------------------- convenience wrapper

def chunk_prefill(q, k, v, g_log, beta, num_householder, cu_seqlens, scale=None, initial_state=None,
                  output_final_state=False, use_qk_l2norm=False, state_cache=None, state_indices=None,
                  return_chunk_states=False, descriptors=None, out=None):
    """Allocating front end in the Megatron Core argument order.

    Accepts an optional leading batch dim of 1 on q/k/v/g/beta (THD packing).
    Returns (o, final_state or None) or, with return_chunk_states,
    (o, final_state or None, chunk_states, chunk_offsets): chunk_states has the
    capacity row count; rows >= chunk_offsets[N] are unwritten padding.
    """
    squeeze = q.dim() == 4
    if squeeze:
        q, k, v, g_log, beta = q[0], k[0], v[0], g_log[0], beta[0]
    T, Hqk, K = q.shape
    Hv, V = v.shape[1], v.shape[2]
    N = cu_seqlens.shape[0] - 1
    dev = q.device
    o = out if out is not None else torch.empty((T, Hv, V), dtype=q.dtype, device=dev)
    fs = torch.empty((N, Hv, K, V), dtype=torch.float32, device=dev) if output_final_state else None
    cs = None
    if return_chunk_states and descriptors is None:
        descriptors = gdp_build_descriptors(cu_seqlens, num_householder, T)
    ws = torch.empty(max(gdp_workspace_bytes(T, N, num_householder, Hqk, Hv, K, V, q.dtype), 256),
                     dtype=torch.uint8, device=dev)
    if return_chunk_states:
        nt_cap, _ = gdp_descriptor_capacity(T, N, num_householder)
        cs = torch.empty((max(nt_cap, 1), Hv, K, V), dtype=torch.float32, device=dev)
    gdp_chunk_prefill(q, k, v, g_log, beta, num_householder, cu_seqlens, scale or 0.0, initial_state,
                      output_final_state, use_qk_l2norm, state_cache, state_indices, return_chunk_states,
                      o, fs, cs, descriptors, ws)
    if squeeze:
        o = o.unsqueeze(0)
    if return_chunk_states:
        return o, fs, cs, descriptors["chunk_offsets"]
    return o, fs


def recurrent_decode(q, k, v, g_log, beta, num_householder, state_cache, state_indices, scale=None,
                     use_qk_l2norm=False, out=None):
    """Allocating front end of the decode step: returns o [N, Hv, V]; the state
    cache is updated in place."""
    N = q.shape[0]
    Hv, V = v.shape[1], v.shape[2]
    o = out if out is not None else torch.empty((N, Hv, V), dtype=q.dtype, device=q.device)
    gdp_recurrent_decode(q, k, v, g_log, beta, num_householder, scale or 0.0, use_qk_l2norm, state_cache,
                         state_indices, o)
    return o


def chunk_gated_delta_product(q, k, v, g=None, beta=None, num_householder=1, scale=None, initial_state=None,
                              output_final_state=False, cu_seqlens=None, use_qk_l2norm_in_kernel=False,
                              output=None, output_state=None):
    """Allocating front end in the FlashInfer convention (FlashInfer docs,
    "flashinfer.gdp_prefill.chunk_gated_delta_product", parameter list): linear
    decays g (None: no decay), beta (None: ones), V-major states.  Returns
    output, or (output, final_state) when output_final_state."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required (varlen input only)")
    T, Hq, d = q.shape
    Hv = v.shape[1]
    N = cu_seqlens.shape[0] - 1
    dev = q.device
    out = output if output is not None else torch.empty((T, Hv, d), dtype=q.dtype, device=dev)
    fs = None
    if output_final_state:
        fs = output_state if output_state is not None else torch.empty(
            (N, Hv, d, d), dtype=initial_state.dtype if initial_state is not None else torch.float32, device=dev)
    ws = torch.empty(max(gdp_fi_workspace_bytes(T, N, num_householder, Hq, Hv, d, q.dtype, initial_state is not None,
                                                output_final_state), 256), dtype=torch.uint8, device=dev)
    gdp_chunk_gated_delta_product(q, k, v, g, beta, num_householder, scale, initial_state, output_final_state,
                                  cu_seqlens, use_qk_l2norm_in_kernel, out, fs, ws)
    return (out, fs) if output_final_state else out


def chunk_prefill_backward(q, k, v, g_log, beta, num_householder, cu_seqlens, d_o, d_final_state=None, scale=None,
                           initial_state=None, use_qk_l2norm=False):
    """Allocating front end of the gradients: returns a dict of float32 tensors
    dq, dk, dv, dg_log, dbeta and d_initial_state (None without an initial state)."""
    T, Hqk, K = q.shape
    Hk, Hv, V = k.shape[1], v.shape[1], v.shape[2]
    N = cu_seqlens.shape[0] - 1
    n = int(num_householder)
    dev = q.device
    f32 = dict(dtype=torch.float32, device=dev)
    dq, dk = torch.empty((T, Hqk, K), **f32), torch.empty((T * n, Hk, K), **f32)
    dv, dg = torch.empty((T * n, Hv, V), **f32), torch.empty((T, Hv), **f32)
    db = torch.empty((T * n, Hv), **f32)
    ds0 = torch.empty((N, Hv, K, V), **f32) if initial_state is not None else None
    ws = torch.empty(max(gdp_backward_workspace_bytes(T, N, n, Hqk, Hv, K, V, q.dtype), 256), dtype=torch.uint8,
                     device=dev)
    gdp_chunk_prefill_backward(q, k, v, g_log, beta, n, cu_seqlens, scale, initial_state, use_qk_l2norm, d_o,
                               d_final_state, dq, dk, dv, dg, db, ds0, ws)
    return {"dq": dq, "dk": dk, "dv": dv, "dg_log": dg, "dbeta": db, "d_initial_state": ds0}


def gated_scan(x, g_log, cu_seqlens, initial_state=None, output_final_state=False, complement_input=False,
               state_cache=None, state_indices=None, return_checkpoints=False, out=None):
    """Allocating front end of the gated linear recurrence h_t = exp(g_log_t) h_{t-1} + u_t over packed
    sequences (x, g_log [T, D]; u = x, or (1 - exp(g_log)) x with complement_input).  Returns
    (o, final_state or None) or, with return_checkpoints, (o, final_state or None, checkpoints), which
    gated_scan_backward takes.  Rows that no sequence covers are left as they are in `out`."""
    T, D = x.shape
    N = cu_seqlens.shape[0] - 1
    o = out if out is not None else _empty(x)
    fs = _empty(x, (N, D), torch.float32) if output_final_state else None
    cp = None
    if return_checkpoints:
        cp = _empty(x, (-(-T // GDP_SCAN_CHECKPOINT_ROWS), D), torch.float32)
    gdp_gated_scan(x, g_log, cu_seqlens, complement_input, initial_state, output_final_state, state_cache,
                   state_indices, return_checkpoints, o, fs, cp,
                   _workspace(x, gdp_gated_scan_workspace_bytes(T, N, D)))
    return (o, fs, cp) if return_checkpoints else (o, fs)


def gated_scan_decode(x, g_log, state_cache, state_indices, complement_input=False, out=None):
    """Allocating front end of the recurrence's single-token step: returns o [N, D] in x's dtype; the
    state cache [S, D] is updated in place."""
    o = out if out is not None else _empty(x)
    gdp_gated_scan_decode(x, g_log, complement_input, state_cache, state_indices, o)
    return o


def gated_scan_backward(x, g_log, cu_seqlens, d_o, d_final_state=None, initial_state=None, complement_input=False,
                        checkpoints=None, grads_like_inputs=False):
    """Allocating front end of the recurrence's gradients: returns a dict of dx, dg_log (float32, or the
    dtypes of x and g_log with grads_like_inputs) and d_initial_state (float32; None without an initial
    state).  Without the forward call's `checkpoints` the states are formed again first."""
    T, D = x.shape
    N = cu_seqlens.shape[0] - 1
    dx = _empty(x, dtype=None if grads_like_inputs else torch.float32)
    dg = _empty(g_log, dtype=None if grads_like_inputs else torch.float32)
    ds0 = _empty(initial_state) if initial_state is not None else None
    gdp_gated_scan_backward(x, g_log, cu_seqlens, complement_input, initial_state, checkpoints, d_o, d_final_state,
                            dx, dg, ds0, _workspace(x, gdp_gated_scan_backward_workspace_bytes(T, N, D)))
    return {"dx": dx, "dg_log": dg, "d_initial_state": ds0}


def group_norm(x, weight=None, bias=None, gate=None, activation=None, subtract_mean=True, eps=1e-5, out=None):
    """Allocating front end of the group norm over the last dimension of x [T, G, V] (the heads' outputs,
    channels last): act(n) without a gate, n * act(gate) with one; weight and bias [V] or [G, V];
    activation None, "silu" or "sigmoid"; subtract_mean=False is the root mean square norm."""
    y = out if out is not None else _empty(x)
    gdp_group_norm(x, weight, bias, gate, activation, subtract_mean, eps, y)
    return y


def group_norm_backward(x, d_y, weight=None, bias=None, gate=None, activation=None, subtract_mean=True, eps=1e-5):
    """Allocating front end of the group norm's gradients: returns a dict of dx and dgate (x's dtype) and
    dweight and dbias (float32), None where the forward call had none.  dx is what the recurrences'
    backward calls take as d_o."""
    T, G, V = x.shape
    dx = _empty(x)
    dz = _empty(x) if gate is not None else None
    dw, db = (None if p is None else _empty(p, dtype=torch.float32) for p in (weight, bias))
    sums = weight is not None or bias is not None
    gdp_group_norm_backward(x, weight, bias, gate, activation, subtract_mean, eps, d_y, dx, dw, db, dz,
                            _workspace(x, gdp_group_norm_backward_workspace_bytes(T, G, V)) if sums else None)
    return {"dx": dx, "dweight": dw, "dbias": db, "dgate": dz}


def short_conv(x, weight, cu_seqlens, bias=None, activation=None, initial_state=None, output_final_state=False,
               state_cache=None, state_indices=None, out=None):
    """Allocating front end of the short causal convolution over packed sequences (x [T, D], weight [D, W], bias
    [D]; activation None, "silu" or "sigmoid"): y_t = act(bias + sum_j weight[:, j] x_{t-W+1+j}).  States are the
    W - 1 inputs before (initial_state) and at the end of (final state, state_cache) each sequence, [N, W-1, D] in
    x's dtype.  Returns (y, final_state or None).  Rows that no sequence covers are left as they are in `out`."""
    T, D = x.shape
    N = cu_seqlens.shape[0] - 1
    y = out if out is not None else _empty(x)
    fs = _empty(x, (N, weight.shape[1] - 1, D)) if output_final_state else None
    gdp_short_conv(x, weight, bias, activation, cu_seqlens, initial_state, output_final_state, state_cache,
                   state_indices, y, fs)
    return y, fs


def short_conv_decode(x, weight, state_cache, state_indices, bias=None, activation=None, out=None):
    """Allocating front end of the convolution's single-token step: returns y [N, D] in x's dtype; the state cache
    [S, W-1, D] is updated in place."""
    y = out if out is not None else _empty(x)
    gdp_short_conv_decode(x, weight, bias, activation, state_cache, state_indices, y)
    return y


def short_conv_backward(x, weight, cu_seqlens, d_y, bias=None, activation=None, initial_state=None,
                        d_final_state=None):
    """Allocating front end of the convolution's gradients: returns a dict of dx (x's dtype), dweight, dbias (None
    without a bias) and d_initial_state (None without an initial state), these three float32."""
    T, D = x.shape
    N, W = cu_seqlens.shape[0] - 1, weight.shape[1]
    dx, dw = _empty(x), _empty(weight, dtype=torch.float32)
    db = _empty(bias, dtype=torch.float32) if bias is not None else None
    ds0 = _empty(initial_state, dtype=torch.float32) if initial_state is not None else None
    gdp_short_conv_backward(x, weight, bias, activation, cu_seqlens, initial_state, d_y, d_final_state, dx, dw, db,
                            ds0, _workspace(x, gdp_short_conv_backward_workspace_bytes(T, N, D, W)))
    return {"dx": dx, "dweight": dw, "dbias": db, "d_initial_state": ds0}


def selective_scan(u, dt, A, B, C, cu_seqlens, skip=None, gate=None, dt_bias=None, dt_softplus=False,
                   initial_state=None, output_final_state=False, state_cache=None, state_indices=None,
                   return_checkpoints=False, out=None):
    """Allocating front end of the selective state space scan over packed sequences: with delta = dt + dt_bias (its
    softplus with dt_softplus), h_t = exp(delta_t A) h_{t-1} + delta_t u_t B_t per channel and state, and
    o_t = (C_t . h_t + skip u_t) silu(gate_t).  u, gate [T, D], dt [T, D] (float32 or u's dtype), A [D, S] float32,
    B, C [T, G, S], skip, dt_bias [D] float32, states [N, D, S] float32.  Returns (o, final_state or None) or, with
    return_checkpoints, (o, final_state or None, checkpoints), which selective_scan_backward takes.  Rows that no
    sequence covers are left as they are in `out`."""
    T, D = u.shape
    N, G, S = cu_seqlens.shape[0] - 1, B.shape[1], A.shape[1]
    o = out if out is not None else _empty(u)
    fs = _empty(u, (N, D, S), torch.float32) if output_final_state else None
    cp = _empty(u, (T // GDP_SELECT_CHECKPOINT_ROWS + N, S, D), torch.float32) if return_checkpoints else None
    gdp_selective_scan(u, dt, A, B, C, skip, gate, dt_bias, dt_softplus, cu_seqlens, initial_state,
                       output_final_state, state_cache, state_indices, return_checkpoints, o, fs, cp,
                       _workspace(u, gdp_selective_scan_workspace_bytes(T, N, D, G, S)))
    return (o, fs, cp) if return_checkpoints else (o, fs)


def selective_scan_decode(u, dt, A, B, C, state_cache, state_indices, skip=None, gate=None, dt_bias=None,
                          dt_softplus=False, out=None):
    """Allocating front end of the selective scan's single-token step (u, dt, gate [N, D], B, C [N, G, S]): returns
    o [N, D] in u's dtype; the state cache [S', D, S] is updated in place."""
    o = out if out is not None else _empty(u)
    gdp_selective_scan_decode(u, dt, A, B, C, skip, gate, dt_bias, dt_softplus, state_cache, state_indices, o)
    return o


def selective_scan_backward(u, dt, A, B, C, cu_seqlens, d_o, skip=None, gate=None, dt_bias=None, dt_softplus=False,
                            initial_state=None, d_final_state=None, checkpoints=None):
    """Allocating front end of the selective scan's gradients: returns a dict of du, dgate, dB, dC (u's dtype), ddt
    (dt's dtype), dA, dskip, ddt_bias and d_initial_state (float32), None where the forward call had none.  Without
    the forward call's `checkpoints` the states are formed again first."""
    T, D = u.shape
    N, G, S = cu_seqlens.shape[0] - 1, B.shape[1], A.shape[1]
    du, ddt, dA, dB, dC = _empty(u), _empty(dt), _empty(A), _empty(B), _empty(C)
    dskip, dz, dbias, ds0 = (None if t is None else _empty(t) for t in (skip, gate, dt_bias, initial_state))
    gdp_selective_scan_backward(u, dt, A, B, C, skip, gate, dt_bias, dt_softplus, cu_seqlens, initial_state,
                                checkpoints, d_o, d_final_state, du, ddt, dA, dB, dC, dskip, dz, dbias, ds0,
                                _workspace(u, gdp_selective_scan_backward_workspace_bytes(
                                    T, N, D, G, S, checkpoints is not None)))
    return {"du": du, "ddt": ddt, "dA": dA, "dB": dB, "dC": dC, "dskip": dskip, "dgate": dz, "ddt_bias": dbias,
            "d_initial_state": ds0}


def residual_norm(x, y, post_weight=None, pre_weight=None, gate=None, activation=None, post_norm=True, pre_norm=True,
                  residual_scale=1.0, eps=1e-5, out=None):
    """Allocating front end of the norms around a block: with p = y rstd(y) post_weight (y post_weight without
    post_norm), returns r = x + residual_scale act(gate) p, the next residual stream in x's dtype, and
    n = r rstd(r) pre_weight, the next block's input in y's dtype (None without pre_norm).  x, y, gate [T, D],
    weights [D]; activation None, "silu" or "sigmoid" is the gate's.  out=x updates the residual stream in place."""
    r = out if out is not None else _empty(x)
    n = _empty(y) if pre_norm else None
    gdp_residual_norm(x, y, post_weight, pre_weight, gate, activation, post_norm, pre_norm, residual_scale, eps, r, n)
    return r, n


def residual_norm_backward(x, y, d_r, d_n, post_weight=None, pre_weight=None, gate=None, activation=None,
                           post_norm=True, pre_norm=True, residual_scale=1.0, eps=1e-5):
    """Allocating front end of the gradients of residual_norm for d_r (None for zeros) and d_n (None without
    pre_norm): returns a dict of dx (x's dtype), dy and dgate (y's dtype), dpost_weight and dpre_weight (float32),
    None where the forward call had none."""
    T, D = y.shape
    dx, dy = _empty(x), _empty(y)
    dz = _empty(y) if gate is not None else None
    dw, dv = (None if w is None else _empty(w, dtype=torch.float32) for w in (post_weight, pre_weight))
    sums = post_weight is not None or pre_weight is not None
    gdp_residual_norm_backward(x, y, post_weight, pre_weight, gate, activation, post_norm, pre_norm, residual_scale,
                               eps, d_r, d_n, dx, dy, dw, dv, dz,
                               _workspace(y, gdp_residual_norm_backward_workspace_bytes(T, D)) if sums else None)
    return {"dx": dx, "dy": dy, "dgate": dz, "dpost_weight": dw, "dpre_weight": dv}
