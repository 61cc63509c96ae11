"""Python binding of the routed-MoE HIP library (include/routed_moe.h).

Argument marshalling only: each function has the C entry point's name, takes torch
tensors (or raw integer device addresses) for the device buffers, passes their addresses
and the current HIP stream to the library and raises ``MoeError`` on a non-zero status.
Every step of the layer runs in the library's HIP kernels; there is no other
implementation behind these names.  If the shared library has not been built, every call
raises -- nothing falls back to another path.
"""

import ctypes
import os

__all__ = [
    "MoeError", "MoeDims", "library_path", "moe_status_string", "moe_workspace_size",
    "moe_prepared_weights_size", "moe_workspace_layout", "moe_route_workspace_size",
    "moe_quantize_nvfp4", "moe_prepare_weights", "moe_route", "moe_route_v2",
    "MoeRouteOptions", "moe_forward", "moe_forward_timed", "MOE_FORWARD_STAGES",
    "MoeRing", "make_ring", "moe_ring_layout", "moe_ring_init", "moe_ring_acquire",
    "moe_ring_publish", "moe_forward_streamed", "moe_sealed_workspace_size",
    "moe_forward_absorb", "moe_forward_seal", "moe_topk_softmax", "moe_forward_noalloc",
    "moe_rmsnorm", "moe_matvec_nvfp4", "moe_grouped_gemm", "moe_combine",
    "MOE_MATVEC_MAX_TOKENS", "MOE_EPILOGUE_NONE", "MOE_EPILOGUE_SITU",
    "MOE_QUANT_E4M3_ROW_DYNAMIC",
    "MOE_NOALLOC_SCRATCH_BYTES", "MOE_RING_ROUTE",
    "MOE_RING_LAYOUT",
    "MOE_RING_OK", "MOE_RING_CONSUMER_TIMEOUT", "MOE_RING_PRODUCER_TIMEOUT",
    "MOE_QUANT_NONE", "MOE_QUANT_INT8_ROW_DYNAMIC", "MOE_QUANT_NVFP4_G16", "MOE_MAX_TOKENS",
    "EXPORTED",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_PKG, "lib", "libroutedmoe.so")

MOE_QUANT_NONE = 0
MOE_QUANT_INT8_ROW_DYNAMIC = 1
MOE_QUANT_NVFP4_G16 = 2
MOE_QUANT_E4M3_ROW_DYNAMIC = 3
MOE_EPILOGUE_NONE = 0
MOE_EPILOGUE_SITU = 1
MOE_MATVEC_MAX_TOKENS = 64
MOE_MAX_TOKENS = 16384
MOE_FORWARD_STAGES = 5
MOE_NOALLOC_SCRATCH_BYTES = 32 << 20

# Every symbol include/routed_moe.h declares.
EXPORTED = ("moe_status_string", "moe_workspace_size", "moe_prepared_weights_size",
            "moe_workspace_layout", "moe_route_workspace_size", "moe_quantize_nvfp4",
            "moe_prepare_weights", "moe_route", "moe_route_v2", "moe_forward",
            "moe_forward_timed", "moe_ring_layout", "moe_ring_init", "moe_ring_acquire",
            "moe_ring_publish", "moe_forward_streamed", "moe_sealed_workspace_size",
            "moe_forward_absorb", "moe_forward_seal", "moe_topk_softmax",
            "moe_forward_noalloc", "moe_rmsnorm", "moe_matvec_nvfp4", "moe_grouped_gemm",
            "moe_combine")

MOE_RING_ROUTE = 0
MOE_RING_LAYOUT = 1
MOE_RING_OK = 0
MOE_RING_CONSUMER_TIMEOUT = 1
MOE_RING_PRODUCER_TIMEOUT = 2


class MoeError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {_status_text(status)} ({status})")


class MoeDims(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("top_k", ctypes.c_int32)]

    def __init__(self, hidden, inter, num_experts, top_k):
        super().__init__(hidden, inter, num_experts, top_k)


class MoeRouteOptions(ctypes.Structure):
    """moe_route_options_t: the routing primitive's options (defaults: all experts, gather
    index, cumsum histogram, no quant, dropless, no capacity, no row limit)."""
    _fields_ = [(n, ctypes.c_int32) for n in (
        "expert_start", "expert_end", "row_idx_type", "expert_tokens_num_type", "quant_mode",
        "drop_pad_mode", "expert_capacity", "active_num")]

    def __init__(self, expert_start=0, expert_end=0, row_idx_type=0, expert_tokens_num_type=0,
                 quant_mode=-1, drop_pad_mode=0, expert_capacity=-1, active_num=-1):
        super().__init__(expert_start, expert_end, row_idx_type, expert_tokens_num_type,
                         quant_mode, drop_pad_mode, expert_capacity, active_num)


class MoeRing(ctypes.Structure):
    """moe_ring_t: a caller-owned ring of token slots (device memory at `base`)."""
    _fields_ = [("base", ctypes.c_void_p), ("bytes", ctypes.c_size_t),
                ("num_slots", ctypes.c_int32), ("tokens_per_slot", ctypes.c_int32)]


class _RingLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in (
        "x", "expert_ids", "route_weights", "counters", "status", "total")]


class _Layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in (
        "x_codes", "x_scales", "x_dec", "sorted_ids", "sorted_row_idx", "expanded_row_idx",
        "expert_counts", "expert_cumsum", "a_codes", "a_scales", "o_rows", "o_exp", "a_amax",
        "total")]


_lib_handle = None


def _lib():
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(library_path):
            raise RuntimeError(
                f"routed-MoE HIP library not built ({library_path} missing); run "
                "`python -m routed_moe_layer_amd.build` (or __graft_entry__.build())")
        lib = ctypes.CDLL(library_path)
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        st = ctypes.c_int
        sig = {
            "moe_status_string": (ctypes.c_char_p, [st]),
            "moe_workspace_size": (st, [MoeDims, I32, ctypes.c_int, ctypes.POINTER(SZ)]),
            "moe_prepared_weights_size": (st, [MoeDims, ctypes.POINTER(SZ)]),
            "moe_workspace_layout": (st, [MoeDims, I32, ctypes.POINTER(_Layout)]),
            "moe_route_workspace_size": (st, [I32, I32, I32, ctypes.POINTER(SZ)]),
            "moe_quantize_nvfp4": (st, [P, I64, I64, I32, P, P, P, P]),
            "moe_prepare_weights": (st, [MoeDims, P, P, P, P, P, SZ, P]),
            "moe_route": (st, [MoeDims, I32, P, P, ctypes.c_int, P, P, P, P, P, P, P, P, SZ, P]),
            "moe_route_v2": (st, [I32, I32, I32, I32, P, P, P, P,
                                  ctypes.POINTER(MoeRouteOptions), P, P, P, P, P, P, SZ, P]),
            "moe_forward": (st, [MoeDims, I32, P, P, P, P, P, P, P, P, P, P, P, SZ, P, P]),
            "moe_forward_timed": (st, [MoeDims, I32, P, P, P, P, P, P, P, P, P, P, P, SZ, P, P,
                                       ctypes.POINTER(P)]),
            "moe_ring_layout": (st, [MoeDims, I32, I32, ctypes.POINTER(_RingLayout)]),
            "moe_topk_softmax": (st, [I32, I32, I32, P, P, P, P]),
            "moe_ring_init": (st, [MoeDims, ctypes.POINTER(MoeRing), P]),
            "moe_ring_acquire": (st, [MoeDims, ctypes.POINTER(MoeRing), I32, ctypes.c_int,
                                      ctypes.c_uint32, P]),
            "moe_ring_publish": (st, [MoeDims, ctypes.POINTER(MoeRing), I32, ctypes.c_int, P]),
            "moe_forward_streamed": (st, [MoeDims, ctypes.POINTER(MoeRing), I32, I32, I32, P, P,
                                          P, P, P, P, P, ctypes.c_uint32, P, SZ, P, P]),
            "moe_sealed_workspace_size": (st, [MoeDims, I32, ctypes.POINTER(SZ)]),
            "moe_forward_absorb": (st, [MoeDims, ctypes.POINTER(MoeRing), I32, I32, I32, P,
                                        ctypes.c_uint32, P, SZ, P]),
            "moe_forward_seal": (st, [MoeDims, I32, P, P, P, P, P, P, P, SZ, P, P]),
            "moe_rmsnorm": (st, [I32, I32, P, P, P, ctypes.c_float, ctypes.c_int, P, P, P, P, P]),
            "moe_matvec_nvfp4": (st, [I32, I32, I32, P, P, P, P, P, I32, P]),
            "moe_grouped_gemm": (st, [I32, I32, I32, I32, ctypes.c_int, ctypes.c_int, P, P, I32, P,
                                      I32, P, P, P, P, P, P, P]),
            "moe_combine": (st, [I32, I32, I32, I32, P, P, P, P, P, P]),
            "moe_forward_noalloc": (st, [MoeDims, I32, P, P, P, P, P, P, P, P, P, P, P, P]),
        }
        for name, (res, args) in sig.items():
            f = getattr(lib, name)
            f.restype, f.argtypes = res, args
        _lib_handle = lib
    return _lib_handle


def _status_text(status):
    try:
        return _lib().moe_status_string(status).decode()
    except Exception:  # the library itself failed to load
        return "status"


def _check(fn, status):
    if status != 0:
        raise MoeError(fn, status)


def _ptr(t):
    """Device address of a tensor (or an int address; None -> NULL)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _nbytes(t):
    return t.numel() * t.element_size()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def moe_status_string(status):
    return _lib().moe_status_string(status).decode()


def moe_workspace_size(dims, max_tokens, quant=MOE_QUANT_NVFP4_G16):
    n = ctypes.c_size_t()
    _check("moe_workspace_size",
           _lib().moe_workspace_size(dims, max_tokens, quant, ctypes.byref(n)))
    return n.value


def moe_prepared_weights_size(dims):
    n = ctypes.c_size_t()
    _check("moe_prepared_weights_size", _lib().moe_prepared_weights_size(dims, ctypes.byref(n)))
    return n.value


def moe_workspace_layout(dims, T):
    lay = _Layout()
    _check("moe_workspace_layout", _lib().moe_workspace_layout(dims, T, ctypes.byref(lay)))
    return {name: getattr(lay, name) for name, _ in _Layout._fields_}


def moe_route_workspace_size(num_rows, top_k, num_experts):
    n = ctypes.c_size_t()
    _check("moe_route_workspace_size",
           _lib().moe_route_workspace_size(num_rows, top_k, num_experts, ctypes.byref(n)))
    return n.value


def moe_quantize_nvfp4(src, groups, rows_per_group, K, q, codes, scales, stream=None):
    _check("moe_quantize_nvfp4", _lib().moe_quantize_nvfp4(
        _ptr(src), groups, rows_per_group, K, _ptr(q), _ptr(codes), _ptr(scales),
        _stream(stream)))


def moe_prepare_weights(dims, w13, w13_sf, w2, w2_sf, prepared, prepared_bytes=None, stream=None):
    nb = _nbytes(prepared) if prepared_bytes is None else prepared_bytes
    _check("moe_prepare_weights", _lib().moe_prepare_weights(
        dims, _ptr(w13), _ptr(w13_sf), _ptr(w2), _ptr(w2_sf), _ptr(prepared), nb,
        _stream(stream)))


def moe_route(dims, T, x, expert_ids, quant, qx, sorted_expert_ids, sorted_row_idx,
              expanded_row_idx, expert_cumsum, expanded_x, expanded_sf_or_scale, workspace,
              workspace_bytes=None, stream=None):
    nb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    _check("moe_route", _lib().moe_route(
        dims, T, _ptr(x), _ptr(expert_ids), quant, _ptr(qx), _ptr(sorted_expert_ids),
        _ptr(sorted_row_idx), _ptr(expanded_row_idx), _ptr(expert_cumsum), _ptr(expanded_x),
        _ptr(expanded_sf_or_scale), _ptr(workspace), nb, _stream(stream)))


def moe_route_v2(num_rows, hidden, num_experts, top_k, x, expert_idx, options, expanded_x,
                 expanded_row_idx, expert_tokens=None, expanded_scale=None,
                 available_idx_num=None, scale=None, offset=None, workspace=None,
                 workspace_bytes=None, stream=None):
    nb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    _check("moe_route_v2", _lib().moe_route_v2(
        num_rows, hidden, num_experts, top_k, _ptr(x), _ptr(expert_idx), _ptr(scale),
        _ptr(offset), ctypes.byref(options), _ptr(expanded_x), _ptr(expanded_row_idx),
        _ptr(expert_tokens), _ptr(expanded_scale), _ptr(available_idx_num), _ptr(workspace),
        nb, _stream(stream)))


def moe_forward(dims, T, x, expert_ids, route_weights, prepared, qx, alpha1, qa, alpha2,
                situ_beta, situ_linear_beta, workspace, out, workspace_bytes=None, stream=None):
    nb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    _check("moe_forward", _lib().moe_forward(
        dims, T, _ptr(x), _ptr(expert_ids), _ptr(route_weights), _ptr(prepared), _ptr(qx),
        _ptr(alpha1), _ptr(qa), _ptr(alpha2), _ptr(situ_beta), _ptr(situ_linear_beta),
        _ptr(workspace), nb, _ptr(out), _stream(stream)))


def moe_forward_noalloc(dims, T, x, expert_ids, route_weights, prepared, qx, alpha1, qa,
                        alpha2, situ_beta, situ_linear_beta, out, stream=None):
    _check("moe_forward_noalloc", _lib().moe_forward_noalloc(
        dims, T, _ptr(x), _ptr(expert_ids), _ptr(route_weights), _ptr(prepared), _ptr(qx),
        _ptr(alpha1), _ptr(qa), _ptr(alpha2), _ptr(situ_beta), _ptr(situ_linear_beta), _ptr(out),
        _stream(stream)))


def moe_forward_timed(dims, T, x, expert_ids, route_weights, prepared, qx, alpha1, qa, alpha2,
                      situ_beta, situ_linear_beta, workspace, out, events,
                      workspace_bytes=None, stream=None):
    """``events``: a sequence of MOE_FORWARD_STAGES + 1 raw hipEvent_t handles (ints)."""
    nb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    ev = (ctypes.c_void_p * len(events))(*events)
    _check("moe_forward_timed", _lib().moe_forward_timed(
        dims, T, _ptr(x), _ptr(expert_ids), _ptr(route_weights), _ptr(prepared), _ptr(qx),
        _ptr(alpha1), _ptr(qa), _ptr(alpha2), _ptr(situ_beta), _ptr(situ_linear_beta),
        _ptr(workspace), nb, _ptr(out), _stream(stream), ev))


def moe_ring_layout(dims, num_slots, tokens_per_slot):
    lay = _RingLayout()
    _check("moe_ring_layout", _lib().moe_ring_layout(dims, num_slots, tokens_per_slot,
                                                     ctypes.byref(lay)))
    return {n: getattr(lay, n) for n, _ in _RingLayout._fields_}


def make_ring(buffer, num_slots, tokens_per_slot):
    """A MoeRing over a device byte buffer (a tensor or an int address with its size)."""
    if isinstance(buffer, tuple):
        base, nbytes = buffer
    else:
        base, nbytes = buffer.data_ptr(), _nbytes(buffer)
    return MoeRing(base, nbytes, num_slots, tokens_per_slot)


def moe_ring_init(dims, ring, stream=None):
    _check("moe_ring_init", _lib().moe_ring_init(dims, ctypes.byref(ring), _stream(stream)))


def moe_ring_acquire(dims, ring, slot, role, timeout_us=0, stream=None):
    _check("moe_ring_acquire", _lib().moe_ring_acquire(dims, ctypes.byref(ring), slot, role,
                                                       timeout_us, _stream(stream)))


def moe_ring_publish(dims, ring, slot, role, stream=None):
    _check("moe_ring_publish", _lib().moe_ring_publish(dims, ctypes.byref(ring), slot, role,
                                                       _stream(stream)))


def moe_forward_streamed(dims, ring, total_tokens, first_chunk, num_chunks, prepared, qx,
                         alpha1, qa, alpha2, situ_beta, situ_linear_beta, workspace, out,
                         timeout_us=0, workspace_bytes=None, stream=None):
    nb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    _check("moe_forward_streamed", _lib().moe_forward_streamed(
        dims, ctypes.byref(ring), total_tokens, first_chunk, num_chunks, _ptr(prepared), _ptr(qx),
        _ptr(alpha1), _ptr(qa), _ptr(alpha2), _ptr(situ_beta), _ptr(situ_linear_beta),
        timeout_us, _ptr(workspace), nb, _ptr(out), _stream(stream)))


def moe_sealed_workspace_size(dims, total_tokens):
    n = ctypes.c_size_t()
    _check("moe_sealed_workspace_size",
           _lib().moe_sealed_workspace_size(dims, total_tokens, ctypes.byref(n)))
    return n.value


def moe_forward_absorb(dims, ring, total_tokens, first_chunk, num_chunks, qx, workspace,
                       timeout_us=0, workspace_bytes=None, stream=None):
    nb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    _check("moe_forward_absorb", _lib().moe_forward_absorb(
        dims, ctypes.byref(ring), total_tokens, first_chunk, num_chunks, _ptr(qx), timeout_us,
        _ptr(workspace), nb, _stream(stream)))


def moe_forward_seal(dims, total_tokens, prepared, alpha1, qa, alpha2, situ_beta,
                     situ_linear_beta, workspace, out, workspace_bytes=None, stream=None):
    nb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    _check("moe_forward_seal", _lib().moe_forward_seal(
        dims, total_tokens, _ptr(prepared), _ptr(alpha1), _ptr(qa), _ptr(alpha2),
        _ptr(situ_beta), _ptr(situ_linear_beta), _ptr(workspace), nb, _ptr(out),
        _stream(stream)))


def moe_topk_softmax(T, num_experts, top_k, logits, expert_ids, route_weights, stream=None):
    _check("moe_topk_softmax", _lib().moe_topk_softmax(
        T, num_experts, top_k, _ptr(logits), _ptr(expert_ids), _ptr(route_weights),
        _stream(stream)))


# What a buffer of the stages may hold, by the names that _checked's callers use: a text for
# messages and the names of the tensor types.  BF16 is passed as 16-bit patterns too, and codes
# and scales of 8 bits or less as bytes.
_KINDS = {
    "bf16": ("BF16", "bfloat16 int16 uint16"),
    "f32": ("float32", "float32"),
    "i32": ("int32", "int32"),
    "int8": ("int8", "int8 uint8"),
    "e4m3": ("E4M3", "float8_e4m3fn uint8"),
    "nvfp4": ("NVFP4 code bytes", "uint8 int8 float4_e2m1fn_x2"),
    "e4m3_scale": ("E4M3 scales", "uint8 float8_e4m3fn"),
    "byte": ("8 bits", "int8 uint8 float8_e4m3fn"),
}
_kind_types = {}


def _load_types():
    import torch
    _kind_types.update({k: frozenset(getattr(torch, n) for n in names.split() if hasattr(torch, n))
                        for k, (_, names) in _KINDS.items()})
    return _kind_types


def _code_kind(quant):
    """The kind of 8-bit codes that a quantization makes or takes (the library refuses others)."""
    if quant == MOE_QUANT_INT8_ROW_DYNAMIC:
        return "int8"
    return "e4m3" if quant == MOE_QUANT_E4M3_ROW_DYNAMIC else "byte"


def _checked(fn, stream, *buffers):
    """The stream's handle and the addresses of the buffers, which are given as
    (name, tensor, elements, kind), the kind one of _KINDS.

    A tensor is looked at before its address is passed on: of a type of that kind, on the
    stream's GPU (the current one unless the stream says otherwise), contiguous and at least
    that many elements; None and int addresses pass as they are."""
    types, device, out = _kind_types or _load_types(), None, [None]
    for name, t, n, kind in buffers:
        if t is None or isinstance(t, int):
            out.append(t)
            continue
        if t.dtype not in types[kind]:
            raise ValueError(f"{fn}: {name} holds {t.dtype}, not {_KINDS[kind][0]}")
        at = t.get_device()                    # -1 on the host
        if at != device:
            if at < 0:
                raise ValueError(f"{fn}: {name} is not on a GPU")
            if device is not None:
                raise ValueError(f"{fn}: {name} is on GPU {at}, others on GPU {device}")
            device = at
        if not t.is_contiguous():
            raise ValueError(f"{fn}: {name} is not contiguous")
        if t.numel() < n:
            raise ValueError(f"{fn}: {name} holds {t.numel()} elements, not {n}")
        out.append(t.data_ptr())
    out[0] = _stream_on(fn, stream, device)
    return out


def _stream_on(fn, stream, device):
    """The handle of a stream, which has to be on the GPU of the tensors (device) if any: the
    library launches on the current GPU."""
    if stream is None and device is None:
        return _stream(None)
    if device is not None:
        import torch
        if torch.cuda.current_device() != device:
            raise ValueError(f"{fn}: the tensors are on GPU {device}, the current one is GPU "
                             f"{torch.cuda.current_device()}")
        if stream is None:
            # torch.cuda.current_stream() without the stream object it makes on the way
            return torch._C._cuda_getCurrentRawStream(device)
        if not isinstance(stream, int) and stream.device_index != device:
            raise ValueError(f"{fn}: the tensors are on GPU {device}, the stream on GPU "
                             f"{stream.device_index}")
    return _stream(stream)


def moe_rmsnorm(T, H, x, residual, weight, eps, quant, residual_out, y, codes, scales,
                stream=None):
    stream, x, residual, weight, residual_out, y, codes, scales = _checked(
        "moe_rmsnorm", stream, ("x", x, T * H, "bf16"), ("residual", residual, T * H, "bf16"),
        ("weight", weight, H, "bf16"), ("residual_out", residual_out, T * H, "bf16"),
        ("y", y, T * H, "bf16"), ("codes", codes, T * H, _code_kind(quant)),
        ("scales", scales, T, "f32"))
    _check("moe_rmsnorm", _lib().moe_rmsnorm(T, H, x, residual, weight, eps, quant, residual_out,
                                             y, codes, scales, stream))


def moe_matvec_nvfp4(T, N, K, x, codes, scales, alpha, y, out_f32=False, stream=None):
    stream, x, codes, scales, alpha, y = _checked(
        "moe_matvec_nvfp4", stream, ("x", x, T * K, "bf16"), ("codes", codes, N * K // 2, "nvfp4"),
        ("scales", scales, N * K // 16, "e4m3_scale"), ("alpha", alpha, 1, "f32"),
        ("y", y, T * N, "f32" if out_f32 else "bf16"))
    _check("moe_matvec_nvfp4", _lib().moe_matvec_nvfp4(T, N, K, x, codes, scales, alpha, y,
                                                       int(out_f32), stream))


def moe_grouped_gemm(R, N, K, E, x, expert_cumsum, w, out, quant=MOE_QUANT_NONE, x_scale=None,
                     w_scale=None, x_rows=None, row_idx=None, row_div=None, situ=False,
                     situ_beta=None, situ_linear_beta=None, stream=None):
    """``x_rows`` defaults to R; ``row_div`` counts with ``row_idx`` only."""
    x_rows = R if x_rows is None else x_rows
    row_div = 1 if row_idx is None or row_div is None else row_div
    kind, Nw = "bf16" if quant == MOE_QUANT_NONE else _code_kind(quant), 2 * N if situ else N
    (stream, x, x_scale, row_idx, expert_cumsum, w, w_scale, situ_beta, situ_linear_beta,
     out) = _checked(
        "moe_grouped_gemm", stream, ("x", x, x_rows * K, kind),
        ("x_scale", x_scale, x_rows, "f32"), ("row_idx", row_idx, R, "i32"),
        ("expert_cumsum", expert_cumsum, E, "i32"), ("w", w, E * Nw * K, kind),
        ("w_scale", w_scale, E * Nw, "f32"), ("situ_beta", situ_beta, E, "f32"),
        ("situ_linear_beta", situ_linear_beta, E, "f32"), ("out", out, R * N, "bf16"))
    _check("moe_grouped_gemm", _lib().moe_grouped_gemm(
        R, N, K, E, quant, MOE_EPILOGUE_SITU if situ else MOE_EPILOGUE_NONE, x, x_scale, x_rows,
        row_idx, row_div, expert_cumsum, w, w_scale, situ_beta, situ_linear_beta, out,
        stream))


def moe_combine(T, H, k, R, rows, expanded_row_idx, route_weights, add, out, stream=None):
    stream, rows, expanded_row_idx, route_weights, add, out = _checked(
        "moe_combine", stream, ("rows", rows, R * H, "bf16"),
        ("expanded_row_idx", expanded_row_idx, T * k, "i32"),
        ("route_weights", route_weights, T * k, "bf16"), ("add", add, T * H, "bf16"),
        ("out", out, T * H, "bf16"))
    _check("moe_combine", _lib().moe_combine(T, H, k, R, rows, expanded_row_idx, route_weights,
                                             add, out, stream))
