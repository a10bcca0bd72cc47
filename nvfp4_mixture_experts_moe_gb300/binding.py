"""Thin Python binding of the C ABI in ``include/moe_nvfp4.h`` and
``include/moe_block.h``.

Argument marshalling only: every function here takes torch tensors (or None
for a NULL pointer) where the C call takes pointers, passes their device
addresses and the current CUDA stream, and raises ``MoeError`` on a status
other than MOE_OK. All arithmetic runs in the CUDA library; if the library
is missing the first call raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libmoe_nvfp4.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA = 0, 1, 2, 3
MOE_ERR_WORKSPACE, MOE_ERR_TIMEOUT, MOE_ERR_DEVICE = 4, 5, 6
MOE_W4A16, MOE_W4A4, MOE_MXFP4 = 0, 1, 2
MOE_SCALE_QUANT, MOE_SCALE_DEQUANT = 0, 1
MOE_DEBUG_WAIT_LIMIT, MOE_DEBUG_EXTRA_ARRIVALS, MOE_DEBUG_DISABLE_DECODE_FUSED, MOE_DEBUG_DECODE_STAGE_KB = 1, 2, 3, 4
MOE_DEBUG_FP4_TILE = 5
MOE_DEBUG_F16_TILE = 6

_lib = None


class MoeError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}"
                         + (f" ({last_cuda_error()})" if status == MOE_ERR_CUDA else ""))


class MoeLayerDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("H", ctypes.c_int), ("I", ctypes.c_int),
                ("I_shared", ctypes.c_int), ("E", ctypes.c_int), ("k", ctypes.c_int),
                ("mode", ctypes.c_int),
                ("w13", ctypes.c_void_p), ("w2", ctypes.c_void_p),
                ("w13_shared", ctypes.c_void_p), ("w2_shared", ctypes.c_void_p),
                ("w_router", ctypes.c_void_p),
                ("x_global_scale", ctypes.c_float), ("h_global_scale", ctypes.c_float),
                ("expert_offset", ctypes.c_int), ("local_experts", ctypes.c_int)]


class MoeGemmArgs(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int), ("gate_up", ctypes.c_int), ("num_groups", ctypes.c_int),
                ("N", ctypes.c_int), ("K", ctypes.c_int),
                ("weights", ctypes.c_void_p), ("last_weights", ctypes.c_void_p),
                ("group_offsets", ctypes.c_void_p), ("a", ctypes.c_void_p),
                ("a_sf", ctypes.c_void_p), ("a_gs", ctypes.c_void_p),
                ("a_row_index", ctypes.c_void_p), ("row_scale", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("out_amax", ctypes.c_void_p), ("rows", ctypes.c_int)]


class MoeKv4Cache(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int), ("page_tokens", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("k_gs", ctypes.c_float), ("v_gs", ctypes.c_float),
                ("pool", ctypes.c_void_p)]


class MoeKv4AttnArgs(ctypes.Structure):
    _fields_ = [("cache", MoeKv4Cache), ("batch", ctypes.c_int), ("q_heads", ctypes.c_int),
                ("total_q", ctypes.c_int), ("max_q", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("q", ctypes.c_void_p), ("q_stride", ctypes.c_longlong), ("cu_q", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("scale", ctypes.c_float),
                ("causal", ctypes.c_int), ("window", ctypes.c_int), ("out", ctypes.c_void_p),
                ("lse", ctypes.c_void_p)]


class MoeKvStepArgs(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("page_tokens", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("tokens", ctypes.c_int), ("free_capacity", ctypes.c_int),
                ("ctx_len", ctypes.c_void_p), ("new_len", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("free_pages", ctypes.c_void_p), ("free_count", ctypes.c_void_p),
                ("free_count_out", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("cu_q", ctypes.c_void_p),
                ("slots", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("device_status", ctypes.c_void_p)]


class MoeBlockNormArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("H", ctypes.c_int),
                ("x", ctypes.c_void_p), ("x_stride", ctypes.c_longlong),
                ("gate", ctypes.c_void_p), ("gate_stride", ctypes.c_longlong),
                ("residual", ctypes.c_void_p), ("residual_stride", ctypes.c_longlong),
                ("residual_f32", ctypes.c_int), ("w_post", ctypes.c_void_p), ("w_pre", ctypes.c_void_p),
                ("residual_scale", ctypes.c_float), ("branch_scale", ctypes.c_float), ("eps", ctypes.c_float),
                ("w_offset", ctypes.c_float), ("residual_out", ctypes.c_void_p), ("out", ctypes.c_void_p)]


class MoeRopePlan(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int), ("axes", ctypes.c_int), ("adjacent", ctypes.c_int),
                ("scale", ctypes.c_float), ("turns", ctypes.c_void_p)]


class MoeRopeArgs(ctypes.Structure):
    _fields_ = [("plan", MoeRopePlan), ("tokens", ctypes.c_int), ("head_dim", ctypes.c_int), ("q_heads", ctypes.c_int),
                ("k_heads", ctypes.c_int), ("inverse", ctypes.c_int),
                ("q", ctypes.c_void_p), ("q_stride", ctypes.c_longlong), ("k", ctypes.c_void_p),
                ("k_stride", ctypes.c_longlong), ("positions", ctypes.c_void_p), ("q_out", ctypes.c_void_p),
                ("q_out_stride", ctypes.c_longlong), ("k_out", ctypes.c_void_p), ("k_out_stride", ctypes.c_longlong)]


class MoeKv4AppendRopeArgs(ctypes.Structure):
    _fields_ = [("cache", MoeKv4Cache), ("plan", MoeRopePlan), ("tokens", ctypes.c_int), ("q_heads", ctypes.c_int),
                ("q", ctypes.c_void_p), ("q_stride", ctypes.c_longlong), ("k", ctypes.c_void_p),
                ("k_stride", ctypes.c_longlong), ("v", ctypes.c_void_p), ("v_stride", ctypes.c_longlong),
                ("slots", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("q_out", ctypes.c_void_p),
                ("q_out_stride", ctypes.c_longlong), ("device_status", ctypes.c_void_p)]


class MoeKv4Index(ctypes.Structure):
    _fields_ = [("cache", MoeKv4Cache), ("block_tokens", ctypes.c_int), ("means", ctypes.c_void_p),
                ("owners", ctypes.c_void_p)]


class MoeKv4SelectArgs(ctypes.Structure):
    _fields_ = [("index", MoeKv4Index), ("batch", ctypes.c_int), ("q_heads", ctypes.c_int), ("total_q", ctypes.c_int),
                ("max_q", ctypes.c_int), ("max_pages", ctypes.c_int), ("q", ctypes.c_void_p),
                ("q_stride", ctypes.c_longlong), ("cu_q", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("top", ctypes.c_int), ("sink", ctypes.c_int), ("local", ctypes.c_int),
                ("blocks", ctypes.c_void_p), ("device_status", ctypes.c_void_p)]


class MoeKv4SparseArgs(ctypes.Structure):
    _fields_ = [("cache", MoeKv4Cache), ("block_tokens", ctypes.c_int), ("batch", ctypes.c_int), ("q_heads", ctypes.c_int),
                ("total_q", ctypes.c_int), ("max_q", ctypes.c_int), ("max_pages", ctypes.c_int), ("top", ctypes.c_int),
                ("q", ctypes.c_void_p), ("q_stride", ctypes.c_longlong), ("cu_q", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("blocks", ctypes.c_void_p),
                ("scale", ctypes.c_float), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("device_status", ctypes.c_void_p)]


_P = ctypes.c_void_p
_I = ctypes.c_int
_Z = ctypes.c_size_t
_SIGS = {
    "moe_status_string": (ctypes.c_char_p, [_I]),
    "moe_last_cuda_error": (ctypes.c_char_p, []),
    "moe_route_topk": (_I, [_P, _I, _I, _I, _P, _P, _P]),
    "moe_router_gemm": (_I, [_P, _P, _I, _I, _I, _P, _P]),
    "moe_nvfp4_quantize_static": (_I, [_P, _I, _I, ctypes.c_float, _P, _P, _P]),
    "moe_mxfp4_quantize": (_I, [_P, _I, _I, _P, _P, _P]),
    "moe_import_global_scale": (_I, [ctypes.c_float, _I, ctypes.POINTER(ctypes.c_float)]),
    "moe_nvfp4_fold_scales": (_I, [_P, _Z, ctypes.c_float, _P, _P]),
    "moe_permute_workspace_size": (_Z, [_I, _I, _I]),
    "moe_permute": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P, _Z, _P]),
    "moe_quantize_workspace_size": (_Z, []),
    "moe_nvfp4_quantize": (_I, [_P, _I, _I, _P, _P, _P, _P, _Z, _P]),
    "moe_prepare_size": (_Z, [_I, _I, _I, _I]),
    "moe_nvfp4_prepare_weights": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P]),
    "moe_gemm_workspace_size": (_Z, [_I]),
    "moe_gemm_workspace_size_rows": (_Z, [_I, _I, _I]),
    "moe_nvfp4_grouped_gemm": (_I, [ctypes.POINTER(MoeGemmArgs), _P, _Z, _P]),
    "moe_swiglu": (_I, [_P, _I, _I, _P, _P]),
    "moe_combine": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _P]),
    "moe_workspace_size": (_Z, [ctypes.POINTER(MoeLayerDesc)]),
    "moe_nvfp4_forward": (_I, [ctypes.POINTER(MoeLayerDesc), _P, _P, _P, _P, _P, _Z, _P]),
    "moe_get_device_status": (_I, [_P, _P]),
    "moe_set_stage_events": (_I, [ctypes.POINTER(ctypes.c_void_p), _I]),
    "moe_kernel_launches": (ctypes.c_ulonglong, []),
    "moe_permute_noalloc": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "moe_debug_set": (_I, [_I, ctypes.c_longlong]),
    "moe_kv4_pool_size": (_Z, [_I, _I, _I, _I]),
    # argument structs: a byref() or the bytes of one (PACK_*)
    "moe_kv4_append": (_I, [_P, _P, _P, ctypes.c_longlong, ctypes.c_longlong, _P, _I, _P, _P]),
    "moe_kv4_read": (_I, [_P, _P, _I, _P, _P, _P, _P]),
    "moe_kv4_attention_workspace_size": (_Z, [_P]),
    "moe_kv4_attention": (_I, [_P, _P, _Z, _P]),
    "moe_kv_step": (_I, [_P, _P]),
    "moe_block_norm": (_I, [_P, _P]),
    "moe_rope_turns": (_I, [_P, _P, _I, _P]),
    "moe_rope": (_I, [_P, _P]),
    "moe_kv4_append_rope": (_I, [_P, _P]),
    "moe_kv4_index_size": (_Z, [_I, _I, _I, _I, _I]),
    "moe_kv4_index_update": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P]),
    "moe_kv4_select": (_I, [_P, _P]),
    "moe_kv4_sparse_attention": (_I, [_P, _P]),
}

# The same structs as bytes: for a call per layer and token, filling a ctypes
# struct field by field costs more than the launch.
PACK_KV4_ATTN = struct.Struct("@4i2fP5iPqPPPfiiPP")
PACK_KV_STEP = struct.Struct("@5i11P")
PACK_BLOCK_NORM = struct.Struct("@iiPqPqPqiPPffffPP")
PACK_ROPE = struct.Struct("@3ifP5iPqPqPPqPq")
PACK_KV4_APPEND_ROPE = struct.Struct("@4i2fP3ifP2iPqPqPqPPPqP")
PACK_KV4_SELECT = struct.Struct("@4i2fPiPP5iPqPPP3iPP")
PACK_KV4_SPARSE = struct.Struct("@4i2fP7iPqPPPPfPPP")

MOE_KV4_WS_ZERO = 4096  # leading workspace bytes of moe_kv4_attention that start at zero

MOE_STAGE_COUNT = 8
STAGES = ["route", "permute", "quantize_x", "gemm1_gate_up_swiglu", "quantize_h", "gemm2_down",
          "combine"]


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"CUDA library not built: {LIB_PATH} is missing "
                               "(run nvfp4_mixture_experts_moe_gb300.build.build())")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def status_string(s):
    return lib().moe_status_string(int(s)).decode()


def last_cuda_error():
    return lib().moe_last_cuda_error().decode()


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if type(stream) is int:
        return stream
    if stream is None:
        if torch.cuda.is_initialized():  # the handle alone: building a Stream object takes longer than a launch
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(status, what):
    if status != MOE_OK:
        raise MoeError(status, what)


def moe_route_topk(logits, T, E, k, topk_ids, topk_w, stream=None):
    _check(lib().moe_route_topk(_ptr(logits), T, E, k, _ptr(topk_ids), _ptr(topk_w), _stream(stream)),
           "moe_route_topk")


def moe_router_gemm(x, w_router, T, H, E, logits, stream=None):
    _check(lib().moe_router_gemm(_ptr(x), _ptr(w_router), T, H, E, _ptr(logits), _stream(stream)),
           "moe_router_gemm")


def moe_permute_workspace_size(T, k, E):
    return lib().moe_permute_workspace_size(T, k, E)


def moe_permute(topk_ids, T, k, E, counts, offsets, perm, inv_perm, ws, stream=None):
    _check(lib().moe_permute(_ptr(topk_ids), T, k, E, _ptr(counts), _ptr(offsets), _ptr(perm),
                             _ptr(inv_perm), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "moe_permute")


def moe_quantize_workspace_size():
    return lib().moe_quantize_workspace_size()


def moe_nvfp4_quantize(x, rows, K, q, sf, gs_out, ws, stream=None):
    _check(lib().moe_nvfp4_quantize(_ptr(x), rows, K, _ptr(q), _ptr(sf), _ptr(gs_out), _ptr(ws),
                                    ws.numel() * ws.element_size(), _stream(stream)),
           "moe_nvfp4_quantize")


def moe_nvfp4_quantize_static(x, rows, K, gs, q, sf, stream=None):
    _check(lib().moe_nvfp4_quantize_static(_ptr(x), rows, K, float(gs), _ptr(q), _ptr(sf), _stream(stream)),
           "moe_nvfp4_quantize_static")


def moe_mxfp4_quantize(x, rows, K, q, sf, stream=None):
    _check(lib().moe_mxfp4_quantize(_ptr(x), rows, K, _ptr(q), _ptr(sf), _stream(stream)), "moe_mxfp4_quantize")


def moe_import_global_scale(stored, fmt):
    """A checkpoint's stored global scale -> the quant-convention gs (host only)."""
    out = ctypes.c_float(0.0)
    _check(lib().moe_import_global_scale(float(stored), int(fmt), ctypes.byref(out)), "moe_import_global_scale")
    return out.value


def moe_nvfp4_fold_scales(sf_in, n, ratio, sf_out, stream=None):
    _check(lib().moe_nvfp4_fold_scales(_ptr(sf_in), n, float(ratio), _ptr(sf_out), _stream(stream)),
           "moe_nvfp4_fold_scales")


def moe_prepare_size(N, K, mode, gate_up):
    return lib().moe_prepare_size(N, K, mode, gate_up)


def moe_nvfp4_prepare_weights(codes, sf, gs, N, K, mode, gate_up, out, stream=None):
    """``gs`` is a sequence of host floats (one, or gate and up); None for MXFP4."""
    gp = None
    if gs is not None:
        arr = (ctypes.c_float * len(gs))(*[float(v) for v in gs])
        gp = ctypes.cast(arr, ctypes.c_void_p)
    _check(lib().moe_nvfp4_prepare_weights(_ptr(codes), _ptr(sf), gp, N, K, mode, gate_up, _ptr(out),
                                           _stream(stream)),
           "moe_nvfp4_prepare_weights")


def moe_gemm_workspace_size(num_groups):
    return lib().moe_gemm_workspace_size(num_groups)


def moe_gemm_workspace_size_rows(num_groups, rows, K):
    return lib().moe_gemm_workspace_size_rows(num_groups, rows, K)


def moe_nvfp4_grouped_gemm(args: MoeGemmArgs, ws, stream=None):
    _check(lib().moe_nvfp4_grouped_gemm(ctypes.byref(args), _ptr(ws), ws.numel() * ws.element_size(),
                                        _stream(stream)),
           "moe_nvfp4_grouped_gemm")


def moe_swiglu(gu, rows, I, h, stream=None):
    _check(lib().moe_swiglu(_ptr(gu), rows, I, _ptr(h), _stream(stream)), "moe_swiglu")


def moe_combine(y, inv_perm, topk_w, y_shared, T, k, H, out, stream=None):
    _check(lib().moe_combine(_ptr(y), _ptr(inv_perm), _ptr(topk_w), _ptr(y_shared), T, k, H, _ptr(out),
                             _stream(stream)),
           "moe_combine")


def moe_workspace_size(desc: MoeLayerDesc):
    return lib().moe_workspace_size(ctypes.byref(desc))


def moe_nvfp4_forward(desc: MoeLayerDesc, x, logits, out, topk_ids_out, ws, stream=None, ws_bytes=None):
    nbytes = ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes
    _check(lib().moe_nvfp4_forward(ctypes.byref(desc), _ptr(x), _ptr(logits), _ptr(out), _ptr(topk_ids_out),
                                   _ptr(ws), nbytes, _stream(stream)),
           "moe_nvfp4_forward")


def moe_get_device_status(ws, stream=None):
    """Synchronises and returns (and clears) the device status word of ``ws``."""
    return lib().moe_get_device_status(_ptr(ws), _stream(stream))


def moe_set_stage_events(events):
    """``events``: list of MOE_STAGE_COUNT torch.cuda.Event (or None to clear)."""
    if events is None:
        _check(lib().moe_set_stage_events(None, 0), "moe_set_stage_events")
        return
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _check(lib().moe_set_stage_events(arr, len(events)), "moe_set_stage_events")


def moe_kernel_launches():
    return int(lib().moe_kernel_launches())


def moe_permute_noalloc(topk_ids, T, k, E, counts, offsets, perm, inv_perm, device_status=None, stream=None):
    """moe_permute without a workspace (fixed device scratch inside the library)."""
    _check(lib().moe_permute_noalloc(_ptr(topk_ids), T, k, E, _ptr(counts), _ptr(offsets), _ptr(perm),
                                     _ptr(inv_perm), _ptr(device_status), _stream(stream)),
           "moe_permute_noalloc")


def moe_debug_set(key, value):
    """Test hook (process-wide): see MOE_DEBUG_* in include/moe_nvfp4.h."""
    _check(lib().moe_debug_set(int(key), int(value)), "moe_debug_set")


def moe_kv4_pool_size(num_pages, page_tokens, kv_heads, head_dim):
    return lib().moe_kv4_pool_size(num_pages, page_tokens, kv_heads, head_dim)


def _arg(a):
    return a if isinstance(a, bytes) else ctypes.byref(a)


def moe_kv4_append(cache, k, v, k_stride, v_stride, slots, tokens, device_status=None, stream=None):
    st = lib().moe_kv4_append(_arg(cache), _ptr(k), _ptr(v), k_stride, v_stride, _ptr(slots), tokens,
                              _ptr(device_status), _stream(stream))
    _check(st, "moe_kv4_append")


def moe_kv4_read(cache, slots, n, k_out, v_out, device_status=None, stream=None):
    st = lib().moe_kv4_read(_arg(cache), _ptr(slots), n, _ptr(k_out), _ptr(v_out), _ptr(device_status),
                            _stream(stream))
    _check(st, "moe_kv4_read")


def moe_kv4_attention_workspace_size(args):
    return lib().moe_kv4_attention_workspace_size(_arg(args))


def moe_kv4_attention(args, ws, stream=None):
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().moe_kv4_attention(_arg(args), _ptr(ws), nbytes, _stream(stream)), "moe_kv4_attention")


def moe_kv_step(args, stream=None):
    _check(lib().moe_kv_step(_arg(args), _stream(stream)), "moe_kv_step")


def moe_block_norm(args, stream=None):
    _check(lib().moe_block_norm(_arg(args), _stream(stream)), "moe_block_norm")


def moe_rope_turns(inv_freq, axis):
    """The entries of a rotation's table (host only): whole numbers of 64 bits."""
    n = len(inv_freq)
    out = (ctypes.c_uint64 * n)()
    _check(lib().moe_rope_turns((ctypes.c_double * n)(*inv_freq), (ctypes.c_int32 * n)(*axis), n, out), "moe_rope_turns")
    return list(out)


def moe_rope(args, stream=None):
    _check(lib().moe_rope(_arg(args), _stream(stream)), "moe_rope")


def moe_kv4_append_rope(args, stream=None):
    _check(lib().moe_kv4_append_rope(_arg(args), _stream(stream)), "moe_kv4_append_rope")


def moe_kv4_index_size(num_pages, page_tokens, kv_heads, head_dim, block_tokens):
    return lib().moe_kv4_index_size(num_pages, page_tokens, kv_heads, head_dim, block_tokens)


def moe_kv4_index_update(index, batch, max_q, max_pages, cu_q, kv_len, block_table, device_status=None, stream=None):
    _check(lib().moe_kv4_index_update(_arg(index), batch, max_q, max_pages, _ptr(cu_q), _ptr(kv_len), _ptr(block_table),
                                      _ptr(device_status), _stream(stream)), "moe_kv4_index_update")


def moe_kv4_select(args, stream=None):
    _check(lib().moe_kv4_select(_arg(args), _stream(stream)), "moe_kv4_select")


def moe_kv4_sparse_attention(args, stream=None):
    _check(lib().moe_kv4_sparse_attention(_arg(args), _stream(stream)), "moe_kv4_sparse_attention")
