"""Thin Python binding of libmxfp4_moe.so (include/mxfp4_moe.h).

Argument marshalling only: each function checks dtypes, contiguity and
devices of the torch tensors it is given, then passes their device pointers,
the sizes and the current HIP stream to the C entry point of the same name.
Every step of the computation runs in the library's HIP kernels; there is no
fallback.  If the library is missing, the first call raises.
"""
from __future__ import annotations

import ctypes

import numpy as np
import os
from typing import Optional

import torch

MXFP4_OK = 0
MXFP4_PATH_AUTO, MXFP4_PATH_GEMV, MXFP4_PATH_GEMM = 0, 1, 2
MXFP4_ROUTE_ERR_ID_RANGE, MXFP4_ROUTE_ERR_ID_DUP = 1, 2
MXFP4_MAX_EXPERTS, MXFP4_MAX_TOPK = 512, 32
MXFP4_DECODE_MAX_EXPERTS, MXFP4_DECODE_MAX_K, MXFP4_GEMM_MAX_K = 64, 3072, 8192
MXFP4_NOALLOC_SCRATCH_BYTES = 128 << 20
MXFP4_DTYPE_BF16, MXFP4_DTYPE_F32 = 0, 1
MOE_NORM_MAX_N, MOE_MAX_TOKENS, MOE_MAX_SEQUENCES = 16384, 1 << 30, 1 << 20

#: the C entry points this binding uses (all declared in include/mxfp4_moe.h)
ENTRY_POINTS = (
    "mxfp4_status_string",
    "mxfp4_last_error",
    "mxfp4_moe_route_group",
    "mxfp4_expert_proj_workspace_size",
    "mxfp4_expert_proj",
    "mxfp4_expert_proj_swiglu",
    "moe_combine",
    "mxfp4_moe_decode",
    "mxfp4_dequantize",
    "mxfp4_moe_dense_route",
    "mxfp4_moe_router",
    "mxfp4_moe_decode_swiglu",
    "mxfp4_expert_proj_combine",
    "mxfp4_expert_proj_noalloc",
    "mxfp4_expert_proj_combine_routed",
    "mxfp4_moe_decode_batch",
    "mxfp4_moe_decode_batch_swiglu",
    "moe_norm",
    "moe_norm_backward_workspace_size",
    "moe_norm_backward",
    "moe_combine_norm",
    "moe_combine_norm_backward_workspace_size",
    "moe_combine_norm_backward",
    "moe_balance_workspace_size",
    "moe_balance",
    "moe_route_backward",
    "mxfp4_quantize",
    "mxfp4_quantize_transposed",
    "mxfp4_matmul",
    "mxfp4_expert_matmul",
    "mxfp4_expert_matmul_swiglu",
    "mxfp4_moe_layer_workspace_size",
    "mxfp4_moe_layer",
)

_lib_handle = None


def library_path() -> str:
    """The in-tree libmxfp4_moe.so, or the build named by MXFP4_MOE_LIB (the
    host-sanitizer build of the same sources, for the ABI tests)."""
    return os.environ.get("MXFP4_MOE_LIB") or os.path.join(os.path.dirname(os.path.abspath(__file__)),
                                                           "libmxfp4_moe.so")


class MXFP4Error(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{_status_text(status)} ({status}): {detail}")
        self.status = status


def load_library():
    """Load libmxfp4_moe.so and declare the C signatures (raises if it is not built)."""
    global _lib_handle
    if _lib_handle is not None:
        return _lib_handle
    path = library_path()
    if not os.path.exists(path):
        raise ImportError(f"{path} is not built; run `python -m mxfp4_mixture_experts_amd.build_lib`")
    lib = ctypes.CDLL(path)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.mxfp4_status_string.argtypes = [i32]
    lib.mxfp4_status_string.restype = ctypes.c_char_p
    lib.mxfp4_last_error.argtypes = []
    lib.mxfp4_last_error.restype = ctypes.c_char_p
    lib.mxfp4_moe_route_group.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp, vp, vp, vp]
    lib.mxfp4_moe_route_group.restype = i32
    lib.mxfp4_expert_proj_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    lib.mxfp4_expert_proj_workspace_size.restype = sz
    lib.mxfp4_expert_proj.argtypes = [vp, vp, vp, i32, i32, i32, vp, i32, i32, i32, vp, vp, vp, i32, vp, sz, vp]
    lib.mxfp4_expert_proj_noalloc.argtypes = [vp, vp, vp, i32, i32, i32, vp, i32, i32, i32, vp, vp, vp, i32, vp]
    lib.mxfp4_expert_proj_noalloc.restype = i32
    lib.mxfp4_expert_proj.restype = i32
    lib.mxfp4_expert_proj_swiglu.argtypes = [vp, vp, vp, i32, i32, i32, vp, i32, i32, i32, vp, vp, vp, i32, vp, sz, vp]
    lib.mxfp4_expert_proj_swiglu.restype = i32
    lib.moe_combine.argtypes = [vp, vp, i32, i32, i32, vp, vp]
    lib.moe_combine.restype = i32
    lib.mxfp4_moe_decode.argtypes = [vp, i32, i32, vp, vp, vp, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp, vp]
    lib.mxfp4_moe_decode.restype = i32
    lib.mxfp4_dequantize.argtypes = [vp, vp, ctypes.c_longlong, i32, vp, vp]
    lib.mxfp4_dequantize.restype = i32
    lib.mxfp4_moe_dense_route.argtypes = [vp, i32, i32, i32, vp, vp]
    lib.mxfp4_moe_dense_route.restype = i32
    lib.mxfp4_moe_router.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp]
    lib.mxfp4_moe_router.restype = i32
    lib.mxfp4_moe_decode_swiglu.argtypes = [vp, i32, i32, vp, vp, vp, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.mxfp4_moe_decode_swiglu.restype = i32
    lib.mxfp4_moe_decode_batch.argtypes = [vp, i32, i32, i32, vp, vp, vp, i32, i32, vp, i32, vp, vp, vp, vp, vp,
                                           vp, vp]
    lib.mxfp4_moe_decode_batch.restype = i32
    lib.mxfp4_moe_decode_batch_swiglu.argtypes = [vp, i32, i32, i32, vp, vp, vp, i32, i32, vp, vp, vp, vp, vp, vp,
                                                  vp, vp]
    lib.mxfp4_moe_decode_batch_swiglu.restype = i32
    lib.mxfp4_expert_proj_combine.argtypes = [vp, vp, vp, i32, i32, i32, vp, i32, i32, vp, vp, vp, vp, vp]
    lib.mxfp4_expert_proj_combine.restype = i32
    lib.mxfp4_expert_proj_combine_routed.argtypes = [vp, vp, vp, i32, i32, i32, vp, i32, i32, i32, vp, vp, vp, vp,
                                                     vp, vp, i32, vp, sz, vp]
    lib.mxfp4_expert_proj_combine_routed.restype = i32
    f32 = ctypes.c_float
    lib.moe_norm.argtypes = [vp, i32, vp, i32, i32, f32, vp, vp]
    lib.moe_norm_backward_workspace_size.argtypes = [i32, i32]
    lib.moe_norm_backward.argtypes = [vp, vp, i32, vp, vp, i32, i32, f32, vp, vp, vp, sz, vp]
    lib.moe_combine_norm.argtypes = [vp, i32, vp, i32, i32, i32, vp, vp, i32, f32, f32, vp, vp, vp, vp]
    lib.moe_combine_norm_backward_workspace_size.argtypes = [i32, i32]
    lib.moe_combine_norm_backward.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, vp, i32, f32, f32, vp, vp,
                                              vp, vp, vp, vp, sz, vp]
    lib.moe_balance_workspace_size.argtypes = [i32, i32, i32]
    lib.moe_balance.argtypes = [vp, vp, i32, i32, i32, vp, i32, vp, vp, vp, vp, sz, vp]
    lib.moe_route_backward.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp, i32, vp, vp, vp, vp, i32, vp]
    i64 = ctypes.c_longlong
    lib.mxfp4_quantize.argtypes = [vp, i32, i64, i32, vp, vp, vp, vp]
    lib.mxfp4_quantize_transposed.argtypes = [vp, i32, i64, i32, vp, vp, vp, vp]
    lib.mxfp4_matmul.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, vp, i32, vp]
    lib.mxfp4_expert_matmul.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp, i32, i32, i32, vp, vp, vp, i32, vp]
    lib.mxfp4_expert_matmul_swiglu.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp, i32, i32, i32, vp, vp, vp, vp]
    lib.mxfp4_moe_layer_workspace_size.restype = sz
    lib.mxfp4_moe_layer_workspace_size.argtypes = [i32] * 5
    lib.mxfp4_moe_layer.argtypes = [vp, i32, i32, i32, i32, i32, i32, vp, ctypes.c_float, vp, vp, vp, vp, vp, vp, vp, vp,
                                    i32, vp, i32, vp, vp, vp, sz, vp]
    for name in ("mxfp4_quantize", "mxfp4_quantize_transposed", "mxfp4_matmul", "mxfp4_expert_matmul",
                 "mxfp4_expert_matmul_swiglu", "mxfp4_moe_layer"):
        getattr(lib, name).restype = i32
    for name in ("moe_norm", "moe_norm_backward", "moe_combine_norm", "moe_combine_norm_backward", "moe_balance",
                 "moe_route_backward"):
        getattr(lib, name).restype = i32
        if hasattr(lib, name + "_workspace_size"):
            getattr(lib, name + "_workspace_size").restype = sz
    _lib_handle = lib
    return lib


def _status_text(status: int) -> str:
    try:
        return load_library().mxfp4_status_string(status).decode()
    except ImportError:
        return "status"


def _check(status: int):
    if status != MXFP4_OK:
        raise MXFP4Error(status, load_library().mxfp4_last_error().decode())


def _ptr(t: Optional[torch.Tensor], name: str, dtypes, device=None):
    if t is None:
        return None
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor, got {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t.data_ptr()


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_U8 = (torch.uint8,)
_I32 = (torch.int32,)
_F32 = (torch.float32,)


def _stream(stream, device):
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def mxfp4_moe_route_group(logits, ids_in, T: int, E: int, k: int, topk_ids, gates, expert_offsets,
                          sorted_rows, error_word=None, stream=None):
    """Route and group (mxfp4_moe_route_group).  logits [T,E] bf16 or None, ids_in [T,k] i32 or
    None; writes topk_ids [T,k] i32, gates [T,k] f32 (optional), expert_offsets [E+1] i32,
    sorted_rows [T*k] i32 and error_word [1] i32 (optional)."""
    lib = load_library()
    dev = expert_offsets.device
    st = lib.mxfp4_moe_route_group(
        _ptr(logits, "logits", _BF16, dev), _ptr(ids_in, "ids_in", _I32, dev), int(T), int(E), int(k),
        _ptr(topk_ids, "topk_ids", _I32, dev), _ptr(gates, "gates", _F32, dev),
        _ptr(expert_offsets, "expert_offsets", _I32, dev), _ptr(sorted_rows, "sorted_rows", _I32, dev),
        _ptr(error_word, "error_word", _I32, dev), _stream(stream, dev))
    _check(st)


def mxfp4_expert_proj_workspace_size(E: int, N: int, T: int, k: int, K: int, x_per_slot: bool,
                                     path: int = MXFP4_PATH_AUTO) -> int:
    n = load_library().mxfp4_expert_proj_workspace_size(int(E), int(N), int(T), int(k), int(K),
                                                        int(bool(x_per_slot)), int(path))
    if n == ctypes.c_size_t(-1).value:
        raise MXFP4Error(1, "invalid sizes for the workspace query")
    return int(n)


def mxfp4_expert_proj(blocks, scales, bias, E: int, N: int, K: int, x, x_per_slot: bool, T: int, k: int,
                      expert_offsets, sorted_rows, out, path: int = MXFP4_PATH_AUTO, workspace=None,
                      stream=None):
    """The routed expert projection (mxfp4_expert_proj); out [T,k,N] f32 is written in place.
    workspace: a uint8 device tensor of at least mxfp4_expert_proj_workspace_size(...) bytes."""
    lib = load_library()
    dev = out.device
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr = _ptr(workspace, "workspace", _U8, dev)
        ws_bytes = workspace.numel()
    st = lib.mxfp4_expert_proj(
        _ptr(blocks, "blocks", _U8, dev), _ptr(scales, "scales", _U8, dev), _ptr(bias, "bias", _BF16, dev),
        int(E), int(N), int(K), _ptr(x, "x", _BF16, dev), int(bool(x_per_slot)), int(T), int(k),
        _ptr(expert_offsets, "expert_offsets", _I32, dev), _ptr(sorted_rows, "sorted_rows", _I32, dev),
        _ptr(out, "out", _F32, dev), int(path), ws_ptr, ctypes.c_size_t(ws_bytes), _stream(stream, dev))
    _check(st)


def mxfp4_expert_proj_noalloc(blocks, scales, bias, E: int, N: int, K: int, x, x_per_slot: bool, T: int, k: int,
                              expert_offsets, sorted_rows, out, path: int = MXFP4_PATH_AUTO, stream=None):
    """mxfp4_expert_proj with the library's static scratch instead of a workspace
    (mxfp4_expert_proj_noalloc); out [T,k,N] f32 is written in place."""
    lib = load_library()
    dev = out.device
    st = lib.mxfp4_expert_proj_noalloc(
        _ptr(blocks, "blocks", _U8, dev), _ptr(scales, "scales", _U8, dev), _ptr(bias, "bias", _BF16, dev),
        int(E), int(N), int(K), _ptr(x, "x", _BF16, dev), int(bool(x_per_slot)), int(T), int(k),
        _ptr(expert_offsets, "expert_offsets", _I32, dev), _ptr(sorted_rows, "sorted_rows", _I32, dev),
        _ptr(out, "out", _F32, dev), int(path), _stream(stream, dev))
    _check(st)


def mxfp4_expert_proj_swiglu(blocks, scales, bias, E: int, N: int, K: int, x, x_per_slot: bool, T: int, k: int,
                             expert_offsets, sorted_rows, act, path: int = MXFP4_PATH_AUTO, workspace=None,
                             stream=None):
    """The routed gate/up projection through the gated activation (mxfp4_expert_proj_swiglu);
    act [T,k,N/2] bf16 is written in place.  Workspace as for mxfp4_expert_proj."""
    lib = load_library()
    dev = act.device
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr = _ptr(workspace, "workspace", _U8, dev)
        ws_bytes = workspace.numel()
    st = lib.mxfp4_expert_proj_swiglu(
        _ptr(blocks, "blocks", _U8, dev), _ptr(scales, "scales", _U8, dev), _ptr(bias, "bias", _BF16, dev),
        int(E), int(N), int(K), _ptr(x, "x", _BF16, dev), int(bool(x_per_slot)), int(T), int(k),
        _ptr(expert_offsets, "expert_offsets", _I32, dev), _ptr(sorted_rows, "sorted_rows", _I32, dev),
        _ptr(act, "act", _BF16, dev), int(path), ws_ptr, ctypes.c_size_t(ws_bytes), _stream(stream, dev))
    _check(st)


def moe_combine(proj, gates, T: int, k: int, N: int, y, stream=None):
    """y[t,n] = sum_s gates[t,s] * proj[t,s,n] (moe_combine); y [T,N] f32 is overwritten."""
    lib = load_library()
    dev = y.device
    st = lib.moe_combine(_ptr(proj, "proj", _F32, dev), _ptr(gates, "gates", _F32, dev), int(T), int(k), int(N),
                         _ptr(y, "y", _F32, dev), _stream(stream, dev))
    _check(st)


def mxfp4_moe_decode(logits, E: int, k: int, blocks, scales, bias, N: int, K: int, x, x_per_slot: bool,
                     topk_ids, gates, expert_offsets, sorted_rows, out, error_word=None, stream=None):
    """One decode token in one launch (mxfp4_moe_decode): routing and grouping from logits [1,E]
    bf16 and the projection into out [1,k,N] f32, with the same outputs as
    mxfp4_moe_route_group followed by mxfp4_expert_proj."""
    lib = load_library()
    dev = out.device
    st = lib.mxfp4_moe_decode(
        _ptr(logits, "logits", _BF16, dev), int(E), int(k), _ptr(blocks, "blocks", _U8, dev),
        _ptr(scales, "scales", _U8, dev), _ptr(bias, "bias", _BF16, dev), int(N), int(K), _ptr(x, "x", _BF16, dev),
        int(bool(x_per_slot)), _ptr(topk_ids, "topk_ids", _I32, dev), _ptr(gates, "gates", _F32, dev),
        _ptr(expert_offsets, "expert_offsets", _I32, dev), _ptr(sorted_rows, "sorted_rows", _I32, dev),
        _ptr(error_word, "error_word", _I32, dev), _ptr(out, "out", _F32, dev), _stream(stream, dev))
    _check(st)


def mxfp4_moe_decode_swiglu(logits, E: int, k: int, blocks, scales, bias, N: int, K: int, x, topk_ids, gates,
                            expert_offsets, sorted_rows, act, error_word=None, stream=None):
    """One decode token through the gate/up projection and the gated activation in one launch
    (mxfp4_moe_decode_swiglu): act [1,k,N/2] bf16, with the same outputs as
    mxfp4_moe_route_group followed by mxfp4_expert_proj_swiglu."""
    lib = load_library()
    dev = act.device
    st = lib.mxfp4_moe_decode_swiglu(
        _ptr(logits, "logits", _BF16, dev), int(E), int(k), _ptr(blocks, "blocks", _U8, dev),
        _ptr(scales, "scales", _U8, dev), _ptr(bias, "bias", _BF16, dev), int(N), int(K), _ptr(x, "x", _BF16, dev),
        _ptr(topk_ids, "topk_ids", _I32, dev), _ptr(gates, "gates", _F32, dev),
        _ptr(expert_offsets, "expert_offsets", _I32, dev), _ptr(sorted_rows, "sorted_rows", _I32, dev),
        _ptr(error_word, "error_word", _I32, dev), _ptr(act, "act", _BF16, dev), _stream(stream, dev))
    _check(st)


def mxfp4_moe_decode_batch(logits, T: int, E: int, k: int, blocks, scales, bias, N: int, K: int, x,
                           x_per_slot: bool, topk_ids, gates, expert_offsets, sorted_rows, out, error_word=None,
                           stream=None):
    """Up to 64 decode tokens in one launch (mxfp4_moe_decode_batch): routing and grouping from
    logits [T,E] bf16 and the projection into out [T,k,N] f32, with the same outputs as
    mxfp4_moe_route_group followed by mxfp4_expert_proj on the GEMV path."""
    lib = load_library()
    dev = out.device
    st = lib.mxfp4_moe_decode_batch(
        _ptr(logits, "logits", _BF16, dev), int(T), int(E), int(k), _ptr(blocks, "blocks", _U8, dev),
        _ptr(scales, "scales", _U8, dev), _ptr(bias, "bias", _BF16, dev), int(N), int(K), _ptr(x, "x", _BF16, dev),
        int(bool(x_per_slot)), _ptr(topk_ids, "topk_ids", _I32, dev), _ptr(gates, "gates", _F32, dev),
        _ptr(expert_offsets, "expert_offsets", _I32, dev), _ptr(sorted_rows, "sorted_rows", _I32, dev),
        _ptr(error_word, "error_word", _I32, dev), _ptr(out, "out", _F32, dev), _stream(stream, dev))
    _check(st)


def mxfp4_moe_decode_batch_swiglu(logits, T: int, E: int, k: int, blocks, scales, bias, N: int, K: int, x,
                                  topk_ids, gates, expert_offsets, sorted_rows, act, error_word=None, stream=None):
    """Up to 64 decode tokens through the gate/up projection and the gated activation in one
    launch (mxfp4_moe_decode_batch_swiglu): act [T,k,N/2] bf16, with the same outputs as
    mxfp4_moe_route_group followed by mxfp4_expert_proj_swiglu on the GEMV path."""
    lib = load_library()
    dev = act.device
    st = lib.mxfp4_moe_decode_batch_swiglu(
        _ptr(logits, "logits", _BF16, dev), int(T), int(E), int(k), _ptr(blocks, "blocks", _U8, dev),
        _ptr(scales, "scales", _U8, dev), _ptr(bias, "bias", _BF16, dev), int(N), int(K), _ptr(x, "x", _BF16, dev),
        _ptr(topk_ids, "topk_ids", _I32, dev), _ptr(gates, "gates", _F32, dev),
        _ptr(expert_offsets, "expert_offsets", _I32, dev), _ptr(sorted_rows, "sorted_rows", _I32, dev),
        _ptr(error_word, "error_word", _I32, dev), _ptr(act, "act", _BF16, dev), _stream(stream, dev))
    _check(st)


def mxfp4_dequantize(blocks, scales, out, stream=None):
    """MXFP4 -> bf16 (mxfp4_dequantize): blocks [..., KB, 16] u8 and scales [..., KB] u8 into
    out [..., KB * 32] bf16 (written in place), in the same layout."""
    lib = load_library()
    dev = out.device
    KB = int(blocks.shape[-2])
    if tuple(blocks.shape[:-1]) != tuple(scales.shape) or blocks.shape[-1] != 16:
        raise ValueError("blocks must be [..., KB, 16] and scales [..., KB]")
    if tuple(out.shape) != tuple(scales.shape[:-1]) + (KB * 32,):
        raise ValueError("out must be [..., KB * 32]")
    rows = int(np.prod(scales.shape[:-1])) if scales.dim() > 1 else 1
    st = lib.mxfp4_dequantize(_ptr(blocks, "blocks", _U8, dev), _ptr(scales, "scales", _U8, dev),
                              ctypes.c_longlong(rows), KB * 32, _ptr(out, "out", _BF16, dev), _stream(stream, dev))
    _check(st)


def mxfp4_moe_dense_route(logits, T: int, E: int, k: int, probs, stream=None):
    """Dense router weights (mxfp4_moe_dense_route): probs [T,E] f32, zero outside each token's top k."""
    lib = load_library()
    dev = probs.device
    st = lib.mxfp4_moe_dense_route(_ptr(logits, "logits", _BF16, dev), int(T), int(E), int(k),
                                   _ptr(probs, "probs", _F32, dev), _stream(stream, dev))
    _check(st)


def mxfp4_moe_router(x, w, bias, T: int, H: int, E: int, logits, stream=None):
    """Router logits (mxfp4_moe_router): logits [T,E] bf16 = x [T,H] . w [E,H]^T + bias [E]."""
    lib = load_library()
    dev = logits.device
    st = lib.mxfp4_moe_router(_ptr(x, "x", _BF16, dev), _ptr(w, "w", _BF16, dev), _ptr(bias, "bias", _BF16, dev),
                              int(T), int(H), int(E), _ptr(logits, "logits", _BF16, dev), _stream(stream, dev))
    _check(st)


def mxfp4_expert_proj_combine(blocks, scales, bias, E: int, N: int, K: int, x, x_per_slot: bool, k: int, topk_ids,
                              gates, y, out=None, stream=None):
    """One token through its k experts and the gate-weighted combine in one launch
    (mxfp4_expert_proj_combine): y [1,N] f32 (and out [1,k,N] f32 if given), equal to
    mxfp4_expert_proj followed by moe_combine."""
    lib = load_library()
    dev = y.device
    st = lib.mxfp4_expert_proj_combine(
        _ptr(blocks, "blocks", _U8, dev), _ptr(scales, "scales", _U8, dev), _ptr(bias, "bias", _BF16, dev), int(E),
        int(N), int(K), _ptr(x, "x", _BF16, dev), int(bool(x_per_slot)), int(k), _ptr(topk_ids, "topk_ids", _I32, dev),
        _ptr(gates, "gates", _F32, dev), _ptr(out, "out", _F32, dev), _ptr(y, "y", _F32, dev), _stream(stream, dev))
    _check(st)


def mxfp4_expert_proj_combine_routed(blocks, scales, bias, E: int, N: int, K: int, x, x_per_slot: bool, T: int,
                                     k: int, topk_ids, gates, expert_offsets, sorted_rows, out, y,
                                     path: int = MXFP4_PATH_AUTO, workspace=None, stream=None):
    """The routed projection of T tokens and the gate-weighted combine
    (mxfp4_expert_proj_combine_routed): out [T,k,N] f32 and y [T,N] f32, equal to
    mxfp4_expert_proj followed by moe_combine; the combine is fused into the
    grouped GEMM.  workspace: as for mxfp4_expert_proj."""
    lib = load_library()
    dev = y.device
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr = _ptr(workspace, "workspace", _U8, dev)
        ws_bytes = workspace.numel()
    st = lib.mxfp4_expert_proj_combine_routed(
        _ptr(blocks, "blocks", _U8, dev), _ptr(scales, "scales", _U8, dev), _ptr(bias, "bias", _BF16, dev),
        int(E), int(N), int(K), _ptr(x, "x", _BF16, dev), int(bool(x_per_slot)), int(T), int(k),
        _ptr(topk_ids, "topk_ids", _I32, dev), _ptr(gates, "gates", _F32, dev),
        _ptr(expert_offsets, "expert_offsets", _I32, dev), _ptr(sorted_rows, "sorted_rows", _I32, dev),
        _ptr(out, "out", _F32, dev), _ptr(y, "y", _F32, dev), int(path), ws_ptr, ctypes.c_size_t(ws_bytes),
        _stream(stream, dev))
    _check(st)


# ---------------------------------------------------------------------------
# The norms around the block and the routing's balance
# ---------------------------------------------------------------------------

# element types by dtype code (bf16 also as its bit patterns, as everywhere in this binding)
_ELEMENTS = {MXFP4_DTYPE_BF16: _BF16, MXFP4_DTYPE_F32: _F32}


def _dtype(t: torch.Tensor, name: str) -> int:
    for code, dtypes in _ELEMENTS.items():
        if t.dtype in dtypes:
            return code
    raise TypeError(f"{name}: dtype {t.dtype} not in {_BF16 + _F32}")


def _arg(t: Optional[torch.Tensor], name: str, dtypes, count: int, device: int):
    """A device pointer, or None: the tensor's type, its contiguous layout, its device (an
    ordinal) and that it holds at least `count` elements."""
    if t is None:
        return None
    if t.dtype in dtypes and t.get_device() == device and t.numel() >= count and t.is_contiguous():
        return t.data_ptr()
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, expected a device tensor on cuda:{device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} holds {t.numel()} elements, {count} needed")


def _sizes32(*sizes: int):
    """Refuse a size that does not fit the C int that it is passed as: the call would see its lower
    half.  (A call looks here only where a size has a bit from the 31st on.)"""
    for v in sizes:
        if not -0x80000000 <= v <= 0x7fffffff:
            raise MXFP4Error(1, f"size {v} does not fit an int32")


def _device_of(t: torch.Tensor, name: str) -> int:
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{name} must be a device tensor, got {t.device}")
    return device


#: the current stream's handle without a Stream object around it, and the current device
#: without the check that the runtime has started (1.1 us less a call of about 5)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _run(entry, device: int, stream, *args):
    """The C entry point on `device` (made current for the call) and its stream."""
    if stream is None and _raw_stream is not None:
        handle = _raw_stream(device)
    else:
        handle = _stream(stream, device)
    if device == _current_device():
        st = entry(*args, handle)
    else:
        with torch.cuda.device(device):
            st = entry(*args, handle)
    if st != MXFP4_OK:
        _check(st)


def _size(n: int, what: str) -> int:
    if n == ctypes.c_size_t(-1).value:
        raise MXFP4Error(1, f"invalid sizes for the {what} workspace query")
    return int(n)


def _workspace(workspace, device: int):
    if workspace is None:
        return None, 0
    return _arg(workspace, "workspace", _U8, 0, device), workspace.numel()


def moe_norm(x, w, T: int, N: int, xn, eps: float = 1e-5, stream=None):
    """The block's input norm (moe_norm): xn [T,N] bf16 = x * rsqrt(mean(x^2) + eps) * w of each row
    of x [T,N] bf16 or f32; w [N] bf16."""
    lib = load_library()
    T, N = int(T), int(N)
    if T >> 31 or N >> 31:
        _sizes32(T, N)
    dev = _device_of(xn, "xn")
    xt = _dtype(x, "x")
    _run(lib.moe_norm, dev, stream, _arg(x, "x", _ELEMENTS[xt], T * N, dev), xt,
         _arg(w, "w", _BF16, N, dev), T, N, float(eps), _arg(xn, "xn", _BF16, T * N, dev))


def moe_norm_backward_workspace_size(T: int, N: int) -> int:
    T, N = int(T), int(N)
    _sizes32(T, N)
    return _size(load_library().moe_norm_backward_workspace_size(T, N), "moe_norm_backward")


def moe_norm_backward(dxn, x, w, T: int, N: int, dx, dw=None, dres=None, eps: float = 1e-5, workspace=None,
                      stream=None):
    """The gradients of moe_norm (moe_norm_backward): dx [T,N] of x's type (dres, the residual
    stream's own gradient, added; dx may be dres) and dw [N] f32 (optional).  workspace: a uint8
    device tensor of at least moe_norm_backward_workspace_size(T, N) bytes, for dw."""
    lib = load_library()
    T, N = int(T), int(N)
    if T >> 31 or N >> 31:
        _sizes32(T, N)
    dev = _device_of(dx, "dx")
    ws, nbytes = _workspace(workspace, dev)
    xt = _dtype(x, "x")
    xs = _ELEMENTS[xt]
    _run(lib.moe_norm_backward, dev, stream, _arg(dxn, "dxn", _BF16, T * N, dev), _arg(x, "x", xs, T * N, dev), xt,
         _arg(w, "w", _BF16, N, dev), _arg(dres, "dres", xs, T * N, dev), T, N, float(eps), _arg(dx, "dx", xs, T * N, dev),
         _arg(dw, "dw", _F32, N, dev), ws, nbytes)


def moe_combine_norm(proj, gates, T: int, k: int, N: int, x, x_out, w_post=None, scale: float = 1.0, w_next=None,
                     xn=None, eps: float = 1e-5, stream=None):
    """The block's output (moe_combine_norm): the combine of proj [T,k,N] f32 or bf16 with gates
    [T,k] f32 (None: every gate 1), the output norm (w_post [N] bf16, None: no norm), x_out [T,N] =
    x + scale * that (of x's type, may be x), and with w_next [N] bf16 the next block's input
    norm into xn [T,N] bf16."""
    lib = load_library()
    T, k, N = int(T), int(k), int(N)
    if T >> 31 or k >> 31 or N >> 31:
        _sizes32(T, k, N)
    dev = _device_of(x_out, "x_out")
    pt, xt = _dtype(proj, "proj"), _dtype(x, "x")
    _run(lib.moe_combine_norm, dev, stream, _arg(proj, "proj", _ELEMENTS[pt], T * k * N, dev), pt,
         _arg(gates, "gates", _F32, T * k, dev), T, k, N, _arg(w_post, "w_post", _BF16, N, dev),
         _arg(x, "x", _ELEMENTS[xt], T * N, dev), xt, float(scale), float(eps), _arg(x_out, "x_out", _ELEMENTS[xt], T * N, dev),
         _arg(w_next, "w_next", _BF16, N, dev), _arg(xn, "xn", _BF16, T * N, dev))


def moe_combine_norm_backward_workspace_size(T: int, N: int) -> int:
    T, N = int(T), int(N)
    _sizes32(T, N)
    return _size(load_library().moe_combine_norm_backward_workspace_size(T, N), "moe_combine_norm_backward")


def moe_combine_norm_backward(dx_out, proj, gates, T: int, k: int, N: int, dx=None, dproj=None, dgates=None,
                              w_post=None, dw_post=None, scale: float = 1.0, dxn=None, x_out=None, w_next=None,
                              dw_next=None, eps: float = 1e-5, workspace=None, stream=None):
    """The gradients of moe_combine_norm (moe_combine_norm_backward) for dx_out [T,N] (None: 0) and
    dxn [T,N] bf16 (None: none; else with the stored x_out and w_next): dx [T,N] (may be dx_out),
    dproj [T,k,N] of proj's type, dgates [T,k] f32, dw_post and dw_next [N] f32, each None where it is not
    wanted.  workspace: a uint8 device tensor of at least
    moe_combine_norm_backward_workspace_size(T, N) bytes, for the weights' gradients."""
    lib = load_library()
    T, k, N = int(T), int(k), int(N)
    if T >> 31 or k >> 31 or N >> 31:
        _sizes32(T, k, N)
    dev = _device_of(proj, "proj")
    stream_like = next((t for t in (dx_out, x_out, dx) if t is not None), None)
    if stream_like is None:
        raise ValueError("one of dx_out and dxn (with x_out) must be given")
    pt, xt = _dtype(proj, "proj"), _dtype(stream_like, "the residual stream")
    ps, xs = _ELEMENTS[pt], _ELEMENTS[xt]
    ws, nbytes = _workspace(workspace, dev)
    _run(lib.moe_combine_norm_backward, dev, stream, _arg(dx_out, "dx_out", xs, T * N, dev),
         _arg(dxn, "dxn", _BF16, T * N, dev), _arg(x_out, "x_out", xs, T * N, dev),
         _arg(w_next, "w_next", _BF16, N, dev), _arg(proj, "proj", ps, T * k * N, dev), pt,
         _arg(gates, "gates", _F32, T * k, dev), T, k, N, _arg(w_post, "w_post", _BF16, N, dev), xt, float(scale), float(eps),
         _arg(dx, "dx", xs, T * N, dev), _arg(dproj, "dproj", ps, T * k * N, dev),
         _arg(dgates, "dgates", _F32, T * k, dev), _arg(dw_post, "dw_post", _F32, N, dev),
         _arg(dw_next, "dw_next", _F32, N, dev), ws, nbytes)


def moe_balance_workspace_size(T: int, E: int, S: int = 1) -> int:
    T, E, S = int(T), int(E), int(S)
    _sizes32(T, E, S)
    return _size(load_library().moe_balance_workspace_size(T, E, S), "moe_balance")


def moe_balance(logits, topk_ids, T: int, E: int, k: int, counts, tokens, losses, seq_offsets=None, S: int = 1,
                workspace=None, stream=None):
    """Per-expert counts, the balance loss and the z loss (moe_balance) of logits [T,E] bf16 and
    topk_ids [T,k] i32: counts [S,E] i32, tokens [S+2] i32 (per sequence, their sum, the non-empty
    sequences), losses [2] f32 (balance, z).  seq_offsets [S+1] i32: packed sequences (None: one of
    all T tokens).  workspace: a uint8 device tensor of at least moe_balance_workspace_size(T, E, S)
    bytes."""
    lib = load_library()
    T, E, k, S = int(T), int(E), int(k), int(S)
    if T >> 31 or E >> 31 or k >> 31 or S >> 31:
        _sizes32(T, E, k, S)
    dev = _device_of(counts, "counts")
    ws, nbytes = _workspace(workspace, dev)
    _run(lib.moe_balance, dev, stream, _arg(logits, "logits", _BF16, T * E, dev),
         _arg(topk_ids, "topk_ids", _I32, T * k, dev), T, E, k,
         _arg(seq_offsets, "seq_offsets", _I32, S + 1, dev), S, _arg(counts, "counts", _I32, S * E, dev),
         _arg(tokens, "tokens", _I32, S + 2, dev), _arg(losses, "losses", _F32, 2, dev), ws, nbytes)


def moe_route_backward(logits, topk_ids, gates, dgates, T: int, E: int, k: int, dlogits, seq_offsets=None, S: int = 1,
                       counts=None, tokens=None, dlosses=None, stream=None):
    """The gradient of the router logits (moe_route_backward) into dlogits [T,E] f32 or bf16: through
    the gates [T,k] (dgates [T,k] f32, or None) and through moe_balance's losses (dlosses [2] f32 on
    the device, or None; with it logits, seq_offsets, S, counts and tokens as given to and written by
    moe_balance)."""
    lib = load_library()
    T, E, k, S = int(T), int(E), int(k), int(S)
    if T >> 31 or E >> 31 or k >> 31 or S >> 31:
        _sizes32(T, E, k, S)
    dev = _device_of(dlogits, "dlogits")
    dt = _dtype(dlogits, "dlogits")
    _run(lib.moe_route_backward, dev, stream, _arg(logits, "logits", _BF16, T * E, dev),
         _arg(topk_ids, "topk_ids", _I32, T * k, dev), _arg(gates, "gates", _F32, T * k, dev),
         _arg(dgates, "dgates", _F32, T * k, dev), T, E, k,
         _arg(seq_offsets, "seq_offsets", _I32, S + 1, dev), S, _arg(counts, "counts", _I32, S * E, dev),
         _arg(tokens, "tokens", _I32, S + 2, dev), _arg(dlosses, "dlosses", _F32, 2, dev),
         _arg(dlogits, "dlogits", _ELEMENTS[dt], T * E, dev), dt)


# ---------------------------------------------------------------------------
# MXFP4 quantisation and the products of two MXFP4 operands
# ---------------------------------------------------------------------------


def _quantize(entry, x, outer: int, inner: int, out_rows: int, out_k: int, blocks, scales, values, stream):
    dev = _device_of(blocks, "blocks")
    xt = _dtype(x, "x")
    n = out_rows * out_k
    _run(entry, dev, stream, _arg(x, "x", _ELEMENTS[xt], n, dev), xt, outer, inner,
         _arg(blocks, "blocks", _U8, n // 2, dev), _arg(scales, "scales", _U8, n // 32, dev),
         _arg(values, "values", _BF16, n, dev))


def mxfp4_quantize(x, blocks, scales, values=None, stream=None):
    """x [..., K] bf16 or f32 -> MXFP4 (mxfp4_quantize): blocks [..., K/32, 16] and scales [..., K/32]
    u8, and what they stand for into values [..., K] bf16 (optional)."""
    K = int(x.shape[-1])
    n = x.numel()
    rows = n // K if K else 0
    if K >> 31:
        _sizes32(K)
    _quantize(load_library().mxfp4_quantize, x, rows, K, rows, K, blocks, scales, values, stream)


def mxfp4_quantize_transposed(x, blocks, scales, values=None, stream=None):
    """x [R, C] bf16 or f32 -> MXFP4 of its transpose, blocks along the rows of x
    (mxfp4_quantize_transposed): blocks [C, R/32, 16] and scales [C, R/32] u8, values [C, R] bf16
    (optional)."""
    if x.dim() != 2:
        raise ValueError(f"x must have two dimensions, has {x.dim()}")
    R, C = x.shape
    if C >> 31:
        _sizes32(C)
    _quantize(load_library().mxfp4_quantize_transposed, x, R, C, C, R, blocks, scales, values, stream)


def mxfp4_matmul(a_blocks, a_scales, b_blocks, b_scales, M: int, N: int, K: int, out, bias=None, stream=None):
    """out [M,N] f32 or bf16 = a . b^T + bias (mxfp4_matmul) of a [M,K] and b [N,K] in MXFP4 (blocks
    [..., K/32, 16] and scales [..., K/32] u8); bias [N] bf16 or None."""
    lib = load_library()
    M, N, K = int(M), int(N), int(K)
    if M >> 31 or N >> 31 or K >> 31:
        _sizes32(M, N, K)
    dev = _device_of(out, "out")
    ot = _dtype(out, "out")
    _run(lib.mxfp4_matmul, dev, stream, _arg(a_blocks, "a_blocks", _U8, M * K // 2, dev),
         _arg(a_scales, "a_scales", _U8, M * K // 32, dev), _arg(b_blocks, "b_blocks", _U8, N * K // 2, dev),
         _arg(b_scales, "b_scales", _U8, N * K // 32, dev), _arg(bias, "bias", _BF16, N, dev), M, N, K,
         _arg(out, "out", _ELEMENTS[ot], M * N, dev), ot)


def _expert_args(blocks, scales, bias, E, N, K, x_blocks, x_scales, x_per_slot, T, k, expert_offsets, sorted_rows,
                 dev):
    rows = T * k if x_per_slot else T
    return (_arg(blocks, "blocks", _U8, E * N * K // 2, dev), _arg(scales, "scales", _U8, E * N * K // 32, dev),
            _arg(bias, "bias", _BF16, E * N, dev), E, N, K, _arg(x_blocks, "x_blocks", _U8, rows * K // 2, dev),
            _arg(x_scales, "x_scales", _U8, rows * K // 32, dev), int(bool(x_per_slot)), T, k,
            _arg(expert_offsets, "expert_offsets", _I32, E + 1, dev),
            _arg(sorted_rows, "sorted_rows", _I32, T * k, dev))


def mxfp4_expert_matmul(blocks, scales, bias, E: int, N: int, K: int, x_blocks, x_scales, x_per_slot: bool, T: int,
                        k: int, expert_offsets, sorted_rows, out, stream=None):
    """The routed projection of MXFP4 activations (mxfp4_expert_matmul): out [T,k,N] f32 or bf16;
    x_blocks and x_scales as mxfp4_quantize writes them for x [T,K], or [T,k,K] with x_per_slot."""
    lib = load_library()
    E, N, K, T, k = int(E), int(N), int(K), int(T), int(k)
    if E >> 31 or N >> 31 or K >> 31 or T >> 31 or k >> 31:
        _sizes32(E, N, K, T, k)
    dev = _device_of(out, "out")
    ot = _dtype(out, "out")
    _run(lib.mxfp4_expert_matmul, dev, stream,
         *_expert_args(blocks, scales, bias, E, N, K, x_blocks, x_scales, x_per_slot, T, k, expert_offsets,
                       sorted_rows, dev), _arg(out, "out", _ELEMENTS[ot], T * k * N, dev), ot)


def mxfp4_expert_matmul_swiglu(blocks, scales, bias, E: int, N: int, K: int, x_blocks, x_scales, x_per_slot: bool,
                               T: int, k: int, expert_offsets, sorted_rows, act, stream=None):
    """The same through the gated activation (mxfp4_expert_matmul_swiglu): act [T,k,N/2] bf16."""
    lib = load_library()
    E, N, K, T, k = int(E), int(N), int(K), int(T), int(k)
    if E >> 31 or N >> 31 or K >> 31 or T >> 31 or k >> 31:
        _sizes32(E, N, K, T, k)
    dev = _device_of(act, "act")
    _run(lib.mxfp4_expert_matmul_swiglu, dev, stream,
         *_expert_args(blocks, scales, bias, E, N, K, x_blocks, x_scales, x_per_slot, T, k, expert_offsets,
                       sorted_rows, dev), _arg(act, "act", _BF16, T * k * (N // 2), dev))


def mxfp4_moe_layer_workspace_size(T: int, H: int, E: int, k: int, F: int) -> int:
    T, H, E, k, F = int(T), int(H), int(E), int(k), int(F)
    _sizes32(T, H, E, k, F)
    return _size(load_library().mxfp4_moe_layer_workspace_size(T, H, E, k, F), "mxfp4_moe_layer")


def mxfp4_moe_layer(x, T: int, H: int, E: int, k: int, F: int, router_w, router_b, gu_blocks, gu_scales, gu_bias,
                    down_blocks, down_scales, down_bias, y, w_norm=None, eps: float = 1e-5, residual: bool = False,
                    topk_ids=None, gates=None, workspace=None, stream=None):
    """A whole expert layer for a few tokens (mxfp4_moe_layer): norm (w_norm [H] bf16; None: x is
    normed), router (router_w [E,H], router_b [E] bf16), gate/up [E,2F,H] and down [E,H,F] experts in
    MXFP4 with bf16 biases, combine and with `residual` + x.  x [T,H] bf16 or (with w_norm) f32, y
    [T,H] bf16 or f32, topk_ids [T,k] i32 and gates [T,k] f32 out; the biases, topk_ids and gates may
    be None.  workspace: a uint8 device tensor of at least
    mxfp4_moe_layer_workspace_size(T, H, E, k, F) bytes, 16-byte aligned."""
    lib = load_library()
    T, H, E, k, F = int(T), int(H), int(E), int(k), int(F)
    if T >> 31 or H >> 31 or E >> 31 or k >> 31 or F >> 31:
        _sizes32(T, H, E, k, F)
    dev = _device_of(y, "y")
    xt, yt = _dtype(x, "x"), _dtype(y, "y")
    ws, nbytes = _workspace(workspace, dev)
    _run(lib.mxfp4_moe_layer, dev, stream, _arg(x, "x", _ELEMENTS[xt], T * H, dev), xt, T, H, E, k, F,
         _arg(w_norm, "w_norm", _BF16, H, dev), float(eps), _arg(router_w, "router_w", _BF16, E * H, dev),
         _arg(router_b, "router_b", _BF16, E, dev), _arg(gu_blocks, "gu_blocks", _U8, E * F * H, dev),
         _arg(gu_scales, "gu_scales", _U8, E * F * H // 16, dev), _arg(gu_bias, "gu_bias", _BF16, E * 2 * F, dev),
         _arg(down_blocks, "down_blocks", _U8, E * H * F // 2, dev),
         _arg(down_scales, "down_scales", _U8, E * H * F // 32, dev), _arg(down_bias, "down_bias", _BF16, E * H, dev),
         int(bool(residual)), _arg(y, "y", _ELEMENTS[yt], T * H, dev), yt,
         _arg(topk_ids, "topk_ids", _I32, T * k, dev), _arg(gates, "gates", _F32, T * k, dev), ws, nbytes)
