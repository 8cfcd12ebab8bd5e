"""ctypes binding of ``libmoe_w4a16.so``: the same entry points, argument
marshalling only.

Each wrapper checks the torch tensors it is given (device, dtype, contiguity,
size) so that the C library, which sees only raw pointers, is never handed a
buffer smaller than the shapes imply; then it passes ``data_ptr()`` and the
stream handle through.  Every computation happens in the HIP kernels.  If the
library is missing this module raises at import-use time -- there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import os
import warnings

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_w4a16.so")

MOE_ACT_NONE = 0
MOE_ACT_SWIGLU = 1
MOE_MAX_TOKENS = 1 << 20
MOE_TILED_MIN_TOKENS = 384
MOE_DOWN_COMBINE_MAX_TOKENS = 4
MOE_DECODE_WORKSPACE_BYTES = 131072
MOE_NOALLOC_MAX_TOKENS = 65536
MOE_NOALLOC_WS_BYTES = 82176
ABI_VERSION = 10

STATUS = {0: "MOE_OK", 1: "MOE_ERR_NULL", 2: "MOE_ERR_SHAPE", 3: "MOE_ERR_UNSUPPORTED",
          4: "MOE_ERR_ALIGN", 5: "MOE_ERR_LAUNCH", 6: "MOE_ERR_DEVICE", 7: "MOE_ERR_WORKSPACE"}

# every symbol include/moe_w4a16.h declares
EXPORTS = ("moe_workspace_bytes", "moe_route", "moe_permute", "moe_route_permute", "moe_route_permute_noalloc", "moe_w4a16_grouped_gemm", "moe_row_sums",
           "moe_w4a16_down_combine", "moe_w4a16_decode_token", "moe_w4a16_decode_token_supported", "moe_combine", "moe_w4a16_prepack", "moe_gen_int4_codes", "moe_gen_fp16_scales",
           "moe_mxfp4_grouped_gemm", "moe_mxfp4_prepack", "moe_gen_ue8m0_scales", "moe_mxfp4_decode_token", "moe_w4a8_decode_token",
           "moe_act_quant_fp8", "moe_act_quant_fp8_dequant", "moe_w4a8_grouped_gemm", "moe_fp8_block_gemm", "moe_fp8_prepack",
           "moe_act_quant_int8", "moe_w8a8_packed_bytes", "moe_w8a8_prepack", "moe_w8a8_gemm", "moe_w8a8_linear",
           "moe_w8a8_grouped_gemm", "moe_w8a8_experts", "moe_balance_workspace_bytes", "moe_balance_loss",
           "moe_route_backward", "moe_status_str", "moe_abi_version")


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__("%s -> %s (%s)" % (fn, STATUS.get(status, status), msg))
        self.status = status


class MoeLayerDesc(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("n_routed", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("n_shared", ctypes.c_int32), ("group_size", ctypes.c_int32),
                ("routed_scale", ctypes.c_float)]

    @classmethod
    def make(cls, hidden, inter, n_routed, top_k, n_shared=1, routed_scale=1.0, group_size=128):
        return cls(hidden, inter, n_routed, top_k, n_shared, group_size, routed_scale)

    @property
    def groups(self) -> int:
        return self.n_routed + self.n_shared

    def rows(self, T: int) -> int:
        return T * (self.top_k + self.n_shared)


_lib = None


def lib() -> ctypes.CDLL:
    """Load the HIP library (raises if it has not been built)."""
    global _lib, _at
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libmoe_w4a16.so is not built (run __graft_entry__.build() or "
                               "python w4a16_routed_expert_moe_amd/build.py); there is no fallback")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, u64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint64, ctypes.c_size_t
        D = ctypes.POINTER(MoeLayerDesc)
        sigs = {
            "moe_route": [D, i32, P, P, P, P, P, P, P],
            "moe_permute": [D, i32, P, P, P, P, P, SZ, P],
            "moe_route_permute": [D, i32, P, P, P, P, P, P, P, P, P, P, SZ, P],
            "moe_route_permute_noalloc": [D, i32, P, P, P, P, P, P, P, P, P, P],
            "moe_w4a16_grouped_gemm": [D, i32, P, P, i32, P, i32, i32, P, P, P, i32, P, P],
            "moe_row_sums": [i32, i32, P, P, P],
            "moe_w4a16_down_combine": [D, i32, P, P, P, P, P, P, P, P],
            "moe_w4a16_decode_token": [D, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P],
            "moe_w4a16_decode_token_supported": [D],
            "moe_combine": [D, i32, P, P, P, P, P],
            "moe_w4a16_prepack": [i32, i32, i32, P, P, P],
            "moe_gen_int4_codes": [u64, i32, i32, i32, i32, i32, i32, P, P],
            "moe_gen_fp16_scales": [u64, i32, i32, i32, i32, i32, i32, P, P],
            "moe_mxfp4_grouped_gemm": [D, i32, P, P, i32, i32, i32, P, P, P, i32, P, P],
            "moe_mxfp4_prepack": [i32, i32, i32, P, P, P],
            "moe_mxfp4_decode_token": [D, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P],
            "moe_w4a8_decode_token": [D, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P],
            "moe_gen_ue8m0_scales": [u64, i32, i32, i32, i32, i32, i32, P, P],
            "moe_act_quant_fp8": [i32, i32, P, P, P, P],
            "moe_act_quant_fp8_dequant": [i32, i32, P, P, P, P, P],
            "moe_w4a8_grouped_gemm": [D, i32, P, P, P, i32, i32, i32, P, P, P, i32, P, P],
            "moe_fp8_block_gemm": [i32, i32, i32, P, P, P, P, P, P],
            "moe_fp8_prepack": [i32, i32, P, P, P],
            "moe_act_quant_int8": [i32, i32, P, P, P, P],
            "moe_w8a8_prepack": [i32, i32, i32, P, P, P],
            "moe_w8a8_gemm": [i32, i32, i32, P, P, P, P, P, P],
            "moe_w8a8_linear": [i32, i32, i32, P, P, P, P, P, P, P],
            "moe_w8a8_grouped_gemm": [D, i32, P, P, P, i32, i32, i32, P, P, P, i32, P, P],
            "moe_w8a8_experts": [D, i32, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P],
            "moe_balance_loss": [D, i32, i32, P, P, P, P, ctypes.c_float, P, P, P, P, P, SZ, P],
            "moe_route_backward": [D, i32, i32, P, P, P, P, P, P, P, P, P, P],
        }
        for name, args in sigs.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        L.moe_workspace_bytes.argtypes = [D, i32]
        L.moe_workspace_bytes.restype = ctypes.c_size_t
        L.moe_w8a8_packed_bytes.argtypes = [i32, i32, i32]
        L.moe_w8a8_packed_bytes.restype = ctypes.c_size_t
        L.moe_balance_workspace_bytes.argtypes = [D, i32, i32]
        L.moe_balance_workspace_bytes.restype = ctypes.c_size_t
        L.moe_status_str.argtypes = [ctypes.c_int]
        L.moe_status_str.restype = ctypes.c_char_p
        L.moe_abi_version.argtypes = []
        L.moe_abi_version.restype = ctypes.c_int32
        if L.moe_abi_version() != ABI_VERSION:
            raise RuntimeError("libmoe_w4a16.so has ABI version %d, this binding expects %d (rebuild)"
                               % (L.moe_abi_version(), ABI_VERSION))
        _at = _native_at() or _checked
        _lib = L
    return _lib


def _native_at():
    """The native form of _checked, or None: without _bind.so, or with one built for another Python or torch (it reads
    their objects at the offsets of the headers it was compiled with), the same checks are made in Python."""
    if not os.path.exists(os.path.join(_HERE, "_bind.so")):
        return None
    from .build import bind_built_for
    try:
        from . import _bind
        built_for = _bind.built_for
    except (ImportError, AttributeError) as e:
        built_for = e
    if built_for != bind_built_for():
        warnings.warn("_bind.so is not one for %s (%s), arguments are checked in Python (rebuild)"
                      % (bind_built_for(), built_for))
        return None
    _bind.set_checked(_checked)
    return _bind.at


def _check(fn: str, status: int):
    if status != 0:
        raise MoeError(fn, status, lib().moe_status_str(status).decode())


def _stream(stream, dev=None) -> int:
    if stream is None:  # the current stream's handle, without building a Stream object
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if dev is None else dev)
    if isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    return int(stream)


_Tensor = torch.Tensor


def _ptr(t, name, dtype, numel, optional=False):
    # the common case first: a call checks up to 17 tensors, and a decode
    # step's calls are bound by the host
    if isinstance(t, _Tensor) and t.is_cuda and t.dtype is dtype and t.is_contiguous() and t.numel() >= numel:
        return t.data_ptr()
    if t is None:
        if optional:
            return None
        raise ValueError("%s is required" % name)
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    raise ValueError("%s holds %d elements, needs %d" % (name, t.numel(), numel))


_BF16, _F32, _I32, _I8, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.int8, torch.uint8


def _checked(dev, t, name, dtype, numel, optional=False):
    """_ptr of a tensor that has to be on device dev: the current one, where the library launches."""
    if isinstance(t, _Tensor) and t.get_device() == dev and t.dtype is dtype and t.is_contiguous() and t.numel() >= numel:
        return t.data_ptr()
    p = _ptr(t, name, dtype, numel, optional)
    if p is not None:
        raise ValueError("%s is on device %d, the current device is %d" % (name, t.get_device(), dev))
    return p


_at = _checked  # until lib() puts the native one in its place: the common case at 0.05 us a tensor instead of 0.3


# What the sizes of a call, or-ed, have above 31 bits when each fits an int32
# (all non-negative, or one negative, which the library refuses): ctypes would
# cut a wider one to another size than the tensors are checked for.
_I32_HIGH = (0, -1)


def _wide(fn):
    raise ValueError("%s: a size does not fit 32 bits" % fn)


# ------------------------------------------------------------------ entry points
def moe_route(desc: MoeLayerDesc, T: int, x, w_router, gate_bias, logits, topk_idx, topk_w,
              stream=None):
    if T >> 31 not in _I32_HIGH:
        _wide("moe_route")
    H, E, k = desc.hidden, desc.n_routed, desc.top_k
    _check("moe_route", lib().moe_route(
        ctypes.byref(desc), T, _ptr(x, "x", torch.bfloat16, T * H),
        _ptr(w_router, "w_router", torch.bfloat16, E * H), _ptr(gate_bias, "gate_bias", torch.float32, E),
        _ptr(logits, "logits", torch.float32, T * E), _ptr(topk_idx, "topk_idx", torch.int32, T * k),
        _ptr(topk_w, "topk_w", torch.float32, T * k), _stream(stream)))


def moe_workspace_bytes(desc: MoeLayerDesc, T: int) -> int:
    """Bytes of the workspace moe_permute / moe_route_permute need at T tokens."""
    if T >> 31 not in _I32_HIGH:
        _wide("moe_workspace_bytes")
    return int(lib().moe_workspace_bytes(ctypes.byref(desc), T))


def _ws(ws, name="ws"):
    """(pointer, bytes) of a uint8 device workspace tensor, or (None, 0)."""
    if ws is None:
        return None, 0
    return _ptr(ws, name, torch.uint8, 0), ws.numel()


def moe_permute(desc: MoeLayerDesc, T: int, topk_idx, group_offsets, sorted_token, row_of_slot,
                ws=None, stream=None):
    if T >> 31 not in _I32_HIGH:
        _wide("moe_permute")
    G, R, S = desc.groups, desc.rows(T), desc.top_k + desc.n_shared
    wp, wb = _ws(ws)
    _check("moe_permute", lib().moe_permute(
        ctypes.byref(desc), T, _ptr(topk_idx, "topk_idx", torch.int32, T * desc.top_k),
        _ptr(group_offsets, "group_offsets", torch.int32, G + 1),
        _ptr(sorted_token, "sorted_token", torch.int32, R),
        _ptr(row_of_slot, "row_of_slot", torch.int32, T * S), wp, wb, _stream(stream)))


def moe_route_permute(desc: MoeLayerDesc, T: int, x, w_router, gate_bias, logits, topk_idx, topk_w,
                      group_offsets, sorted_token, row_of_slot, ws, stream=None):
    if T >> 31 not in _I32_HIGH:
        _wide("moe_route_permute")
    H, E, k = desc.hidden, desc.n_routed, desc.top_k
    G, R, S = desc.groups, desc.rows(T), desc.top_k + desc.n_shared
    _check("moe_route_permute", lib().moe_route_permute(
        ctypes.byref(desc), T, _ptr(x, "x", torch.bfloat16, T * H),
        _ptr(w_router, "w_router", torch.bfloat16, E * H), _ptr(gate_bias, "gate_bias", torch.float32, E),
        _ptr(logits, "logits", torch.float32, T * E), _ptr(topk_idx, "topk_idx", torch.int32, T * k),
        _ptr(topk_w, "topk_w", torch.float32, T * k),
        _ptr(group_offsets, "group_offsets", torch.int32, G + 1),
        _ptr(sorted_token, "sorted_token", torch.int32, R),
        _ptr(row_of_slot, "row_of_slot", torch.int32, T * S), *_ws(ws), _stream(stream)))


def moe_route_permute_noalloc(desc: MoeLayerDesc, T: int, x, w_router, gate_bias, logits, topk_idx,
                              topk_w, group_offsets, sorted_token, row_of_slot, stream=None):
    """moe_route_permute with the library's own static scratch (no workspace)."""
    if T >> 31 not in _I32_HIGH:
        _wide("moe_route_permute_noalloc")
    H, E, k = desc.hidden, desc.n_routed, desc.top_k
    G, R, S = desc.groups, desc.rows(T), desc.top_k + desc.n_shared
    _check("moe_route_permute_noalloc", lib().moe_route_permute_noalloc(
        ctypes.byref(desc), T, _ptr(x, "x", torch.bfloat16, T * H),
        _ptr(w_router, "w_router", torch.bfloat16, E * H), _ptr(gate_bias, "gate_bias", torch.float32, E),
        _ptr(logits, "logits", torch.float32, T * E), _ptr(topk_idx, "topk_idx", torch.int32, T * k),
        _ptr(topk_w, "topk_w", torch.float32, T * k),
        _ptr(group_offsets, "group_offsets", torch.int32, G + 1),
        _ptr(sorted_token, "sorted_token", torch.int32, R),
        _ptr(row_of_slot, "row_of_slot", torch.int32, T * S), _stream(stream)))


def moe_w4a16_grouped_gemm(desc: MoeLayerDesc, T: int, a, a_gather, n_src: int, a_sums, N: int, K: int,
                           w_packed, w_scales, group_offsets, act: int, out, stream=None):
    if (T | N | K | act) >> 31 not in _I32_HIGH or n_src >> 31 not in _I32_HIGH:
        _wide("moe_w4a16_grouped_gemm")
    G, R = desc.groups, desc.rows(T)
    a_rows = n_src if a_gather is not None else R
    out_cols = N // 2 if act == MOE_ACT_SWIGLU else N
    _check("moe_w4a16_grouped_gemm", lib().moe_w4a16_grouped_gemm(
        ctypes.byref(desc), T, _ptr(a, "a", torch.bfloat16, a_rows * K),
        _ptr(a_gather, "a_gather", torch.int32, R, optional=True), n_src,
        _ptr(a_sums, "a_sums", torch.float32, a_rows * (K // 128), optional=True), N, K,
        _ptr(w_packed, "w_packed", torch.uint8, G * N * K // 2),
        _ptr(w_scales, "w_scales", torch.float16, G * N * (K // 128)),
        _ptr(group_offsets, "group_offsets", torch.int32, G + 1), act,
        _ptr(out, "out", torch.bfloat16, R * out_cols), _stream(stream)))


def moe_mxfp4_grouped_gemm(desc: MoeLayerDesc, T: int, a, a_gather, n_src: int, N: int, K: int,
                           w_packed, w_scales, group_offsets, act: int, out, stream=None):
    if (T | N | K | act) >> 31 not in _I32_HIGH or n_src >> 31 not in _I32_HIGH:
        _wide("moe_mxfp4_grouped_gemm")
    G, R = desc.groups, desc.rows(T)
    a_rows = n_src if a_gather is not None else R
    out_cols = N // 2 if act == MOE_ACT_SWIGLU else N
    _check("moe_mxfp4_grouped_gemm", lib().moe_mxfp4_grouped_gemm(
        ctypes.byref(desc), T, _ptr(a, "a", torch.bfloat16, a_rows * K),
        _ptr(a_gather, "a_gather", torch.int32, R, optional=True), n_src, N, K,
        _ptr(w_packed, "w_packed", torch.uint8, G * N * K // 2),
        _ptr(w_scales, "w_scales", torch.uint8, G * N * (K // 32)),
        _ptr(group_offsets, "group_offsets", torch.int32, G + 1), act,
        _ptr(out, "out", torch.bfloat16, R * out_cols), _stream(stream)))


def moe_row_sums(rows: int, K: int, a, sums, stream=None):
    if (rows | K) >> 31 not in _I32_HIGH:
        _wide("moe_row_sums")
    _check("moe_row_sums", lib().moe_row_sums(
        rows, K, _ptr(a, "a", torch.bfloat16, rows * K),
        _ptr(sums, "sums", torch.float32, rows * (K // 128)), _stream(stream)))


def moe_w4a16_down_combine(desc: MoeLayerDesc, T: int, h, w_packed, w_scales, topk_idx, topk_w,
                           row_of_slot, out, stream=None):
    if T >> 31 not in _I32_HIGH:
        _wide("moe_w4a16_down_combine")
    H, I, G, R, S = desc.hidden, desc.inter, desc.groups, desc.rows(T), desc.top_k + desc.n_shared
    _check("moe_w4a16_down_combine", lib().moe_w4a16_down_combine(
        ctypes.byref(desc), T, _ptr(h, "h", torch.bfloat16, R * I),
        _ptr(w_packed, "w_packed", torch.uint8, G * H * I // 2),
        _ptr(w_scales, "w_scales", torch.float16, G * H * (I // 128)),
        _ptr(topk_idx, "topk_idx", torch.int32, T * desc.top_k),
        _ptr(topk_w, "topk_w", torch.float32, T * desc.top_k),
        _ptr(row_of_slot, "row_of_slot", torch.int32, T * S),
        _ptr(out, "out", torch.bfloat16, T * H), _stream(stream)))


def moe_w4a16_decode_token(desc: MoeLayerDesc, x, w_router, gate_bias, w13_packed, w13_scales, w2_packed,
                           w2_scales, logits, topk_idx, topk_w, group_offsets, sorted_token, row_of_slot,
                           h, out, workspace, stream=None):
    H, I, E, k = desc.hidden, desc.inter, desc.n_routed, desc.top_k
    G, S = desc.groups, desc.top_k + desc.n_shared
    _check("moe_w4a16_decode_token", lib().moe_w4a16_decode_token(
        ctypes.byref(desc), _ptr(x, "x", torch.bfloat16, H),
        _ptr(w_router, "w_router", torch.bfloat16, E * H), _ptr(gate_bias, "gate_bias", torch.float32, E),
        _ptr(w13_packed, "w13_packed", torch.uint8, G * 2 * I * H // 2),
        _ptr(w13_scales, "w13_scales", torch.float16, G * 2 * I * (H // 128)),
        _ptr(w2_packed, "w2_packed", torch.uint8, G * H * I // 2),
        _ptr(w2_scales, "w2_scales", torch.float16, G * H * (I // 128)),
        _ptr(logits, "logits", torch.float32, E), _ptr(topk_idx, "topk_idx", torch.int32, k),
        _ptr(topk_w, "topk_w", torch.float32, k), _ptr(group_offsets, "group_offsets", torch.int32, G + 1),
        _ptr(sorted_token, "sorted_token", torch.int32, S), _ptr(row_of_slot, "row_of_slot", torch.int32, S),
        _ptr(h, "h", torch.bfloat16, S * I), _ptr(out, "out", torch.bfloat16, H),
        _ptr(workspace, "workspace", torch.int32, MOE_DECODE_WORKSPACE_BYTES // 4), _stream(stream)))


def moe_mxfp4_decode_token(desc: MoeLayerDesc, x, w_router, gate_bias, w13_packed, w13_scales, w2_packed,
                           w2_scales, logits, topk_idx, topk_w, group_offsets, sorted_token, row_of_slot,
                           h, out, workspace, stream=None):
    H, I, E, k = desc.hidden, desc.inter, desc.n_routed, desc.top_k
    G, S = desc.groups, desc.top_k + desc.n_shared
    _check("moe_mxfp4_decode_token", lib().moe_mxfp4_decode_token(
        ctypes.byref(desc), _ptr(x, "x", torch.bfloat16, H),
        _ptr(w_router, "w_router", torch.bfloat16, E * H), _ptr(gate_bias, "gate_bias", torch.float32, E),
        _ptr(w13_packed, "w13_packed", torch.uint8, G * 2 * I * H // 2),
        _ptr(w13_scales, "w13_scales", torch.uint8, G * 2 * I * (H // 32)),
        _ptr(w2_packed, "w2_packed", torch.uint8, G * H * I // 2),
        _ptr(w2_scales, "w2_scales", torch.uint8, G * H * (I // 32)),
        _ptr(logits, "logits", torch.float32, E), _ptr(topk_idx, "topk_idx", torch.int32, k),
        _ptr(topk_w, "topk_w", torch.float32, k), _ptr(group_offsets, "group_offsets", torch.int32, G + 1),
        _ptr(sorted_token, "sorted_token", torch.int32, S), _ptr(row_of_slot, "row_of_slot", torch.int32, S),
        _ptr(h, "h", torch.bfloat16, S * I), _ptr(out, "out", torch.bfloat16, H),
        _ptr(workspace, "workspace", torch.int32, MOE_DECODE_WORKSPACE_BYTES // 4), _stream(stream)))


def moe_w4a8_decode_token(desc: MoeLayerDesc, x, w_router, gate_bias, w13_packed, w13_scales, w2_packed,
                           w2_scales, logits, topk_idx, topk_w, group_offsets, sorted_token, row_of_slot,
                           h, out, workspace, stream=None):
    """moe_mxfp4_decode_token with x and h quantised to e4m3 per 128 for the expert GEMMs (W4A8)."""
    H, I, E, k = desc.hidden, desc.inter, desc.n_routed, desc.top_k
    G, S = desc.groups, desc.top_k + desc.n_shared
    _check("moe_w4a8_decode_token", lib().moe_w4a8_decode_token(
        ctypes.byref(desc), _ptr(x, "x", torch.bfloat16, H),
        _ptr(w_router, "w_router", torch.bfloat16, E * H), _ptr(gate_bias, "gate_bias", torch.float32, E),
        _ptr(w13_packed, "w13_packed", torch.uint8, G * 2 * I * H // 2),
        _ptr(w13_scales, "w13_scales", torch.uint8, G * 2 * I * (H // 32)),
        _ptr(w2_packed, "w2_packed", torch.uint8, G * H * I // 2),
        _ptr(w2_scales, "w2_scales", torch.uint8, G * H * (I // 32)),
        _ptr(logits, "logits", torch.float32, E), _ptr(topk_idx, "topk_idx", torch.int32, k),
        _ptr(topk_w, "topk_w", torch.float32, k), _ptr(group_offsets, "group_offsets", torch.int32, G + 1),
        _ptr(sorted_token, "sorted_token", torch.int32, S), _ptr(row_of_slot, "row_of_slot", torch.int32, S),
        _ptr(h, "h", torch.bfloat16, S * I), _ptr(out, "out", torch.bfloat16, H),
        _ptr(workspace, "workspace", torch.int32, MOE_DECODE_WORKSPACE_BYTES // 4), _stream(stream)))


def moe_w4a16_decode_token_supported(desc: MoeLayerDesc) -> int:
    """The status moe_w4a16_decode_token would return for `desc` on the current device (0 = supported)."""
    return int(lib().moe_w4a16_decode_token_supported(ctypes.byref(desc)))


def moe_combine(desc: MoeLayerDesc, T: int, y, row_of_slot, topk_w, out, stream=None):
    if T >> 31 not in _I32_HIGH:
        _wide("moe_combine")
    H, R, S = desc.hidden, desc.rows(T), desc.top_k + desc.n_shared
    _check("moe_combine", lib().moe_combine(
        ctypes.byref(desc), T, _ptr(y, "y", torch.bfloat16, R * H),
        _ptr(row_of_slot, "row_of_slot", torch.int32, T * S),
        _ptr(topk_w, "topk_w", torch.float32, T * desc.top_k), _ptr(out, "out", torch.bfloat16, T * H),
        _stream(stream)))


def moe_w4a16_prepack(n_groups: int, N: int, K: int, w_canonical, w_packed, stream=None):
    if (n_groups | N | K) >> 31 not in _I32_HIGH:
        _wide("moe_w4a16_prepack")
    n = n_groups * N * K // 2
    _check("moe_w4a16_prepack", lib().moe_w4a16_prepack(
        n_groups, N, K, _ptr(w_canonical, "w_canonical", torch.uint8, n),
        _ptr(w_packed, "w_packed", torch.uint8, n), _stream(stream)))


def moe_mxfp4_prepack(n_groups: int, N: int, K: int, w_canonical, w_packed, stream=None):
    if (n_groups | N | K) >> 31 not in _I32_HIGH:
        _wide("moe_mxfp4_prepack")
    n = n_groups * N * K // 2
    _check("moe_mxfp4_prepack", lib().moe_mxfp4_prepack(
        n_groups, N, K, _ptr(w_canonical, "w_canonical", torch.uint8, n),
        _ptr(w_packed, "w_packed", torch.uint8, n), _stream(stream)))


def moe_gen_ue8m0_scales(seed: int, layer: int, group0: int, n_groups: int, kind: int, N: int, K: int,
                         out, stream=None):
    if (n_groups | N | K) >> 31 not in _I32_HIGH:
        _wide("moe_gen_ue8m0_scales")
    _check("moe_gen_ue8m0_scales", lib().moe_gen_ue8m0_scales(
        seed, layer, group0, n_groups, kind, N, K,
        _ptr(out, "out", torch.uint8, n_groups * N * (K // 32)), _stream(stream)))


def moe_gen_int4_codes(seed: int, layer: int, group0: int, n_groups: int, kind: int, N: int, K: int,
                       out, stream=None):
    if (n_groups | N | K) >> 31 not in _I32_HIGH:
        _wide("moe_gen_int4_codes")
    _check("moe_gen_int4_codes", lib().moe_gen_int4_codes(
        seed, layer, group0, n_groups, kind, N, K,
        _ptr(out, "out", torch.uint8, n_groups * N * K // 2), _stream(stream)))


def moe_gen_fp16_scales(seed: int, layer: int, group0: int, n_groups: int, kind: int, N: int, K: int,
                        out, stream=None):
    if (n_groups | N | K) >> 31 not in _I32_HIGH:
        _wide("moe_gen_fp16_scales")
    _check("moe_gen_fp16_scales", lib().moe_gen_fp16_scales(
        seed, layer, group0, n_groups, kind, N, K,
        _ptr(out, "out", torch.float16, n_groups * N * (K // 128)), _stream(stream)))


def moe_status_str(status: int) -> str:
    return lib().moe_status_str(status).decode()


def moe_abi_version() -> int:
    return lib().moe_abi_version()


# ------------------------------------------------------------------ fp8 activations
def moe_act_quant_fp8(rows: int, K: int, a, codes, scales, stream=None):
    if (rows | K) >> 31 not in _I32_HIGH:
        _wide("moe_act_quant_fp8")
    _check("moe_act_quant_fp8", lib().moe_act_quant_fp8(
        rows, K, _ptr(a, "a", torch.bfloat16, rows * K), _ptr(codes, "codes", torch.uint8, rows * K),
        _ptr(scales, "scales", torch.uint8, rows * (K // 128)), _stream(stream)))


def moe_act_quant_fp8_dequant(rows: int, K: int, a, codes, scales, deq, stream=None):
    if (rows | K) >> 31 not in _I32_HIGH:
        _wide("moe_act_quant_fp8_dequant")
    _check("moe_act_quant_fp8_dequant", lib().moe_act_quant_fp8_dequant(
        rows, K, _ptr(a, "a", torch.bfloat16, rows * K), _ptr(codes, "codes", torch.uint8, rows * K),
        _ptr(scales, "scales", torch.uint8, rows * (K // 128)), _ptr(deq, "deq", torch.bfloat16, rows * K),
        _stream(stream)))


def moe_w4a8_grouped_gemm(desc: MoeLayerDesc, T: int, a, a_scales, a_gather, n_src: int, N: int, K: int,
                          w_packed, w_scales, group_offsets, act: int, out, stream=None):
    if (T | N | K | act) >> 31 not in _I32_HIGH or n_src >> 31 not in _I32_HIGH:
        _wide("moe_w4a8_grouped_gemm")
    G, R = desc.groups, desc.rows(T)
    a_rows = n_src if a_gather is not None else R
    out_cols = N // 2 if act == MOE_ACT_SWIGLU else N
    _check("moe_w4a8_grouped_gemm", lib().moe_w4a8_grouped_gemm(
        ctypes.byref(desc), T, _ptr(a, "a", torch.uint8, a_rows * K),
        _ptr(a_scales, "a_scales", torch.uint8, a_rows * (K // 128)),
        _ptr(a_gather, "a_gather", torch.int32, R, optional=True), n_src, N, K,
        _ptr(w_packed, "w_packed", torch.uint8, G * N * K // 2),
        _ptr(w_scales, "w_scales", torch.uint8, G * N * (K // 32)),
        _ptr(group_offsets, "group_offsets", torch.int32, G + 1), act,
        _ptr(out, "out", torch.bfloat16, R * out_cols), _stream(stream)))


def moe_fp8_block_gemm(M: int, N: int, K: int, a, a_scales, w_packed, w_scales, out, stream=None):
    if (M | N | K) >> 31 not in _I32_HIGH:
        _wide("moe_fp8_block_gemm")
    _check("moe_fp8_block_gemm", lib().moe_fp8_block_gemm(
        M, N, K, _ptr(a, "a", torch.uint8, M * K), _ptr(a_scales, "a_scales", torch.uint8, M * (K // 128)),
        _ptr(w_packed, "w_packed", torch.uint8, N * K),
        _ptr(w_scales, "w_scales", torch.uint8, (N // 128) * (K // 128)),
        _ptr(out, "out", torch.bfloat16, M * N), _stream(stream)))


def moe_fp8_prepack(N: int, K: int, w_canonical, w_packed, stream=None):
    if (N | K) >> 31 not in _I32_HIGH:
        _wide("moe_fp8_prepack")
    _check("moe_fp8_prepack", lib().moe_fp8_prepack(
        N, K, _ptr(w_canonical, "w_canonical", torch.uint8, N * K), _ptr(w_packed, "w_packed", torch.uint8, N * K),
        _stream(stream)))


# ------------------------------------------------------------------ W8A8
def moe_act_quant_int8(rows: int, K: int, a, codes, scales, stream=None):
    if (rows | K) >> 31 not in _I32_HIGH:
        _wide("moe_act_quant_int8")
    d = torch.cuda.current_device()
    _check("moe_act_quant_int8", lib().moe_act_quant_int8(
        rows, K, _at(d, a, "a", _BF16, rows * K), _at(d, codes, "codes", _I8, rows * K),
        _at(d, scales, "scales", _F32, rows), _stream(stream, d)))


def moe_w8a8_packed_bytes(n_groups: int, N: int, K: int) -> int:
    """Bytes of the packed weights of n_groups matrices [N][K] (0 when a size is invalid)."""
    if (n_groups | N | K) >> 31 not in _I32_HIGH:
        _wide("moe_w8a8_packed_bytes")
    return int(lib().moe_w8a8_packed_bytes(n_groups, N, K))


def _packed(n_groups: int, N: int, K: int) -> int:
    """moe_w8a8_packed_bytes of valid sizes, without the call (the entry points refuse the others)."""
    return n_groups * ((N + 63) & -64) * ((K + 127) & -128)


def moe_w8a8_prepack(n_groups: int, N: int, K: int, w_canonical, w_packed, stream=None):
    if (n_groups | N | K) >> 31 not in _I32_HIGH:
        _wide("moe_w8a8_prepack")
    d = torch.cuda.current_device()
    _check("moe_w8a8_prepack", lib().moe_w8a8_prepack(
        n_groups, N, K, _at(d, w_canonical, "w_canonical", _I8, n_groups * N * K),
        _at(d, w_packed, "w_packed", _I8, moe_w8a8_packed_bytes(n_groups, N, K)), _stream(stream, d)))


def moe_w8a8_gemm(M: int, N: int, K: int, a, a_scales, w_packed, w_scales, out, stream=None):
    if (M | N | K) >> 31 not in _I32_HIGH:
        _wide("moe_w8a8_gemm")
    d = torch.cuda.current_device()
    _check("moe_w8a8_gemm", lib().moe_w8a8_gemm(
        M, N, K, _at(d, a, "a", _I8, M * K), _at(d, a_scales, "a_scales", _F32, M),
        _at(d, w_packed, "w_packed", _I8, _packed(1, N, K)),
        _at(d, w_scales, "w_scales", _F32, N), _at(d, out, "out", _BF16, M * N), _stream(stream, d)))


def moe_w8a8_linear(M: int, N: int, K: int, x, w_packed, w_scales, codes, scales, out, stream=None):
    """moe_act_quant_int8 + moe_w8a8_gemm in one call; codes and scales are scratch."""
    if (M | N | K) >> 31 not in _I32_HIGH:
        _wide("moe_w8a8_linear")
    d = torch.cuda.current_device()
    _check("moe_w8a8_linear", lib().moe_w8a8_linear(
        M, N, K, _at(d, x, "x", _BF16, M * K),
        _at(d, w_packed, "w_packed", _I8, _packed(1, N, K)),
        _at(d, w_scales, "w_scales", _F32, N), _at(d, codes, "codes", _I8, M * K),
        _at(d, scales, "scales", _F32, M), _at(d, out, "out", _BF16, M * N), _stream(stream, d)))


def moe_w8a8_grouped_gemm(desc: MoeLayerDesc, T: int, a, a_scales, a_gather, n_src: int, N: int, K: int,
                          w_packed, w_scales, group_offsets, act: int, out, stream=None):
    if (T | N | K | act) >> 31 not in _I32_HIGH or n_src >> 31 not in _I32_HIGH:  # (n_src is not used without a_gather)
        _wide("moe_w8a8_grouped_gemm")
    G, R = desc.groups, desc.rows(T)
    a_rows = n_src if a_gather is not None else R
    out_cols = N // 2 if act == MOE_ACT_SWIGLU else N
    d = torch.cuda.current_device()
    _check("moe_w8a8_grouped_gemm", lib().moe_w8a8_grouped_gemm(
        ctypes.byref(desc), T, _at(d, a, "a", _I8, a_rows * K),
        _at(d, a_scales, "a_scales", _F32, a_rows),
        _at(d, a_gather, "a_gather", _I32, R, True), n_src, N, K,
        _at(d, w_packed, "w_packed", _I8, _packed(G, N, K)),
        _at(d, w_scales, "w_scales", _F32, G * N),
        _at(d, group_offsets, "group_offsets", _I32, G + 1), act,
        _at(d, out, "out", _BF16, R * out_cols), _stream(stream, d)))


def moe_w8a8_experts(desc: MoeLayerDesc, T: int, x, topk_w, group_offsets, sorted_token, row_of_slot, w13_packed,
                     w13_scales, w2_packed, w2_scales, xq, xqs, h, hq, hqs, y, out, stream=None):
    """Everything after the routing for INT8 experts; xq, xqs, hq and hqs are scratch."""
    if T >> 31 not in _I32_HIGH:
        _wide("moe_w8a8_experts")
    H, I, G, R, S = desc.hidden, desc.inter, desc.groups, desc.rows(T), desc.top_k + desc.n_shared
    d = torch.cuda.current_device()
    _check("moe_w8a8_experts", lib().moe_w8a8_experts(
        ctypes.byref(desc), T, _at(d, x, "x", _BF16, T * H),
        _at(d, topk_w, "topk_w", _F32, T * desc.top_k),
        _at(d, group_offsets, "group_offsets", _I32, G + 1),
        _at(d, sorted_token, "sorted_token", _I32, R), _at(d, row_of_slot, "row_of_slot", _I32, T * S),
        _at(d, w13_packed, "w13_packed", _I8, _packed(G, 2 * I, H)),
        _at(d, w13_scales, "w13_scales", _F32, G * 2 * I),
        _at(d, w2_packed, "w2_packed", _I8, _packed(G, H, I)),
        _at(d, w2_scales, "w2_scales", _F32, G * H), _at(d, xq, "xq", _I8, T * H),
        _at(d, xqs, "xqs", _F32, T), _at(d, h, "h", _BF16, R * I),
        _at(d, hq, "hq", _I8, R * I), _at(d, hqs, "hqs", _F32, R),
        _at(d, y, "y", _BF16, R * H), _at(d, out, "out", _BF16, T * H), _stream(stream, d)))


# ------------------------------------------------------------------ router balance and gradient
def moe_balance_workspace_bytes(desc: MoeLayerDesc, T: int, n_seq: int) -> int:
    """Bytes of the workspace moe_balance_loss needs (0 when a size is invalid)."""
    if (T | n_seq) >> 31 not in _I32_HIGH:
        _wide("moe_balance_workspace_bytes")
    return int(lib().moe_balance_workspace_bytes(ctypes.byref(desc), T, n_seq))


def _mask(m):
    """A mask of truth values as the bytes it consists of."""
    return m.view(_U8) if isinstance(m, _Tensor) and m.dtype is torch.bool else m


def moe_balance_loss(desc: MoeLayerDesc, T: int, n_seq: int, seq_offsets, token_mask, logits, topk_idx, alpha: float,
                     counts, prob_sums, seq_coef, loss, ws, stream=None):
    if (T | n_seq) >> 31 not in _I32_HIGH:
        _wide("moe_balance_loss")
    E, k = desc.n_routed, desc.top_k
    d = torch.cuda.current_device()
    _check("moe_balance_loss", lib().moe_balance_loss(
        ctypes.byref(desc), T, n_seq, _at(d, seq_offsets, "seq_offsets", _I32, n_seq + 1, True),
        _at(d, _mask(token_mask), "token_mask", _U8, T, True), _at(d, logits, "logits", _F32, T * E),
        _at(d, topk_idx, "topk_idx", _I32, T * k), alpha, _at(d, counts, "counts", _I32, n_seq * E),
        _at(d, prob_sums, "prob_sums", _F32, n_seq * E), _at(d, seq_coef, "seq_coef", _F32, n_seq),
        _at(d, loss, "loss", _F32, 1), _at(d, ws, "ws", _U8, 0), ws.numel(), _stream(stream, d)))


def moe_route_backward(desc: MoeLayerDesc, T: int, n_seq: int, seq_offsets, token_mask, logits, topk_idx, counts,
                       seq_coef, d_loss, d_topk_w, d_logits, stream=None):
    if (T | n_seq) >> 31 not in _I32_HIGH:
        _wide("moe_route_backward")
    E, k = desc.n_routed, desc.top_k
    d = torch.cuda.current_device()
    _check("moe_route_backward", lib().moe_route_backward(
        ctypes.byref(desc), T, n_seq, _at(d, seq_offsets, "seq_offsets", _I32, n_seq + 1, True),
        _at(d, _mask(token_mask), "token_mask", _U8, T, True), _at(d, logits, "logits", _F32, T * E),
        _at(d, topk_idx, "topk_idx", _I32, T * k),
        _at(d, counts, "counts", _I32, n_seq * E, d_loss is None),
        _at(d, seq_coef, "seq_coef", _F32, n_seq, d_loss is None),
        _at(d, d_loss, "d_loss", _F32, 1, True),
        _at(d, d_topk_w, "d_topk_w", _F32, T * k, True),
        _at(d, d_logits, "d_logits", _F32, T * E), _stream(stream, d)))
