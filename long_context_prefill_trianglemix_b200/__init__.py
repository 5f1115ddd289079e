"""TriangleMix prefill attention on NVIDIA B200 (sm_100a).

Python binding of ``libtm.so`` (C ABI in ``include/tm.h``). The functions named
``tm_*`` take the C ABI's arguments one for one; tensors may be passed as
torch tensors (their ``data_ptr()`` is used) or as raw device addresses.
This module only marshals arguments: every step of the attention runs in the
library's CUDA kernels. PyTorch provides device memory and streams.

If the library has not been built, every call raises; there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import operator
import os
from typing import Any, NamedTuple

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtm.so")

TM_OK, TM_ERR_INVALID_ARG, TM_ERR_UNSUPPORTED, TM_ERR_CUDA, TM_ERR_TIMEOUT = 0, -1, -2, -3, -4
TM_BLOCK_M = TM_BLOCK_N = 128
TM_ROPE_HALF, TM_ROPE_INTERLEAVED = 0, 1
TM_KV_INT8, TM_KV_E4M3 = 0, 1

EXPORTED = (
    "tm_causal_attn_fwd", "tm_triangle_attn_fwd", "tm_trianglemix_attn_fwd",
    "tm_trianglemix_attn_fwd_host",
    "tm_triangle_kept_pairs", "tm_kept_tiles", "tm_triangle_tile_list", "tm_tile_list",
    "tm_debug_dump_tiles", "tm_debug_mma_probe", "tm_debug_schedule", "tm_debug_schedule_window",
    "tm_get_device_status",
    "tm_status_string", "tm_attn_workspace_size", "tm_causal_attn_fwd_ws", "tm_triangle_attn_fwd_ws",
    "tm_trianglemix_attn_fwd_ws", "tm_trianglemix_attn_fwd_noalloc", "tm_block_sparse_attn_fwd",
    "tm_trianglemix_sparse_attn_fwd", "tm_flashprefill_workspace_size",
    "tm_flashprefill_index_capacity", "tm_flashprefill_block_index", "tm_triangle_attn_fwd_heads",
    "tm_debug_inject_stall", "tm_debug_launch_count", "tm_debug_schedule_heads",
    "tm_rope_fwd", "tm_rope_inv_freq", "tm_kv8_append", "tm_kv8_compact",
    "tm_kv8_attn_workspace_size", "tm_kv8_attn_fwd", "tm_key_weights_workspace_size",
    "tm_key_weights_fwd", "tm_kv_select",
)


class TmError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status} ({status_string(status)})")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded ``libtm.so``; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing; build it with "
                "`python -m long_context_prefill_trianglemix_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, ci, cf, cll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong
        cd = ctypes.c_double
        sig = {
            "tm_causal_attn_fwd": (ci, [vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, vp]),
            "tm_triangle_attn_fwd": (ci, [vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, ci, ci, ci, vp]),
            "tm_trianglemix_attn_fwd": (ci, [vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, ci, ci, ci,
                                             ci, ci, vp]),
            "tm_trianglemix_attn_fwd_host": (ci, [vp, vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci,
                                                  ci, cf, ci, ci, ci, ci, ci, ci, vp]),
            "tm_triangle_kept_pairs": (cll, [ci, ci, ci, ci]),
            "tm_kept_tiles": (cll, [ci, ci, ci, ci, ci]),
            "tm_triangle_tile_list": (ci, [ci, ci, ci, ci, ci, ci, vp, cll,
                                           ctypes.POINTER(cll)]),
            "tm_tile_list": (ci, [ci, ci, ci, ci, ci, ci, ci, vp, cll, ctypes.POINTER(cll)]),
            "tm_debug_dump_tiles": (ci, [ci, ci, ci, ci, ci, vp, cll, ctypes.POINTER(cll), vp]),
            "tm_debug_mma_probe": (ci, [vp, vp, vp, vp, vp, ci, vp]),
            "tm_debug_schedule": (ci, [ci, ci, ci, ci, ci, ci, ci, ci, ci, ci, vp, cll,
                                       ctypes.POINTER(cll)]),
            "tm_debug_schedule_window": (ci, [ci, ci, ci, ci, ci, ci, ci, ci, ci, ci, ci, ci, vp,
                                              cll, ctypes.POINTER(cll)]),
            "tm_attn_workspace_size": (ci, [ci, ci, ci, ci, ci, ci, ci, ci, ci, ci,
                                            ctypes.POINTER(cll)]),
            "tm_causal_attn_fwd_ws": (ci, [vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, vp, cll, vp]),
            "tm_triangle_attn_fwd_ws": (ci, [vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, ci, ci, ci,
                                             vp, cll, vp]),
            "tm_trianglemix_attn_fwd_ws": (ci, [vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, ci, ci,
                                                ci, ci, ci, vp, cll, vp]),
            "tm_trianglemix_attn_fwd_noalloc": (ci, [vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, ci,
                                                     ci, ci, ci, ci, vp]),
            "tm_block_sparse_attn_fwd": (ci, [vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, vp, vp, cll,
                                              vp]),
            "tm_trianglemix_sparse_attn_fwd": (ci, [vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, ci, ci,
                                                    ci, ci, ci, vp, vp, cll, vp]),
            "tm_flashprefill_workspace_size": (ci, [ci, ci, ci, ci, ci, ci, ctypes.POINTER(cll)]),
            "tm_triangle_attn_fwd_heads": (ci, [vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, vp, vp, ci,
                                                vp, cll, vp]),
            "tm_flashprefill_index_capacity": (cll, [ci, ci, ci]),
            "tm_flashprefill_block_index": (ci, [vp, vp, ci, ci, ci, ci, ci, cf, cf, ci, vp, cll,
                                                 vp, vp, cll, vp, vp]),
            "tm_get_device_status": (ci, [vp]),
            "tm_debug_inject_stall": (ci, [vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, ci, ci, ci, vp]),
            "tm_status_string": (ctypes.c_char_p, [ci]),
            "tm_debug_launch_count": (cll, []),
            "tm_debug_schedule_heads": (ci, [ci, ci, ci, ci, vp, vp, ci, ci, ci, vp, cll,
                                             ctypes.POINTER(cll)]),
            "tm_rope_fwd": (ci, [vp, vp, vp, vp, ci, ci, ci, ci, ci, cll, cll, cll, cll, ci, ci,
                                 ci, vp, cf, vp, cll, vp]),
            "tm_rope_inv_freq": (ci, [ci, cd, cd, cd, cd, cd, vp]),
            "tm_kv8_append": (ci, [vp, vp, cll, cll, ci, ci, ci, ci, ci, vp, vp, vp, vp, ci, vp,
                                   vp, vp, vp, ci, ci, ci, vp]),
            "tm_kv8_compact": (ci, [vp, ci, vp, vp, ci, ci, ci, vp, ci, vp, ci, vp, vp, vp, vp,
                                    ci, ci, ci, vp, cll, vp, cll, vp]),
            "tm_kv8_attn_workspace_size": (ci, [ci, ci, ci, ci, ci, ci, ci, ci,
                                                ctypes.POINTER(cll)]),
            "tm_kv8_attn_fwd": (ci, [vp, vp, ci, ci, ci, ci, ci, cf, vp, vp, vp, vp, ci, ci, ci,
                                     vp, ci, vp, vp, cll, ci, vp, cll, vp]),
            "tm_key_weights_workspace_size": (ci, [ci, ci, ci, ci, ci, ci, ctypes.POINTER(cll)]),
            "tm_key_weights_fwd": (ci, [vp, vp, ci, ci, ci, ci, ci, cf, ci, vp, vp, cll, ci, vp,
                                        cll, vp]),
            "tm_kv_select": (ci, [vp, cll, vp, ci, ci, ci, ci, ci, ci, vp, vp, vp]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().tm_status_string(int(status)).decode()


def _ptr(x):
    if x is None:
        return None
    try:
        return x.data_ptr()
    except AttributeError:
        return int(x)


_current_stream = None
_device = None


def _find_current_stream():
    """Sets _current_stream and _device, functions that give the handle of torch's current stream
    and the number of its current device; returns the latter. torch.cuda.current_stream() builds
    a Stream object first, 3.3 us of a short call's 10 us on the host; the raw handle (0.2 us) is
    taken where torch gives it."""
    global _current_stream, _device
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    device = getattr(torch._C, "_cuda_getDevice", None)
    torch.cuda.current_stream()  # initialises CUDA
    if raw is None or device is None:
        _current_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
        _device = torch.cuda.current_device
    else:
        _current_stream = lambda: raw(device())  # noqa: E731
        _device = device
    return _device


def _stream(s):
    if s is None:
        if _current_stream is None:
            _find_current_stream()
        return _current_stream()
    if hasattr(s, "cuda_stream"):
        return s.cuda_stream
    return int(s)


def _check(fn: str, rc: int) -> int:
    if rc != TM_OK:
        raise TmError(fn, rc)
    return rc


# ----------------------------------------------------------------------- C ABI, one for one

def tm_causal_attn_fwd(q, k, v, o, B, Hq, Hkv, N, D, scale, stream=None):
    return _check("tm_causal_attn_fwd", lib().tm_causal_attn_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), B, Hq, Hkv, N, D, scale, _stream(stream)))


def tm_triangle_attn_fwd(q, k, v, o, B, Hq, Hkv, N, D, scale, S, W, L, stream=None):
    return _check("tm_triangle_attn_fwd", lib().tm_triangle_attn_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), B, Hq, Hkv, N, D, scale, S, W, L, _stream(stream)))


def tm_trianglemix_attn_fwd(q, k, v, o, B, Hq, Hkv, N, D, scale, S, W, L, layer, tri_start,
                            stream=None):
    return _check("tm_trianglemix_attn_fwd", lib().tm_trianglemix_attn_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), B, Hq, Hkv, N, D, scale, S, W, L, layer, tri_start,
        _stream(stream)))


def tm_trianglemix_attn_fwd_host(q_host, k_host, v_host, o_host, q_dev, k_dev, v_dev, o_dev, B,
                                 Hq, Hkv, N, D, scale, S, W, L, layer, tri_start, chunk_rows=0,
                                 stream=None):
    return _check("tm_trianglemix_attn_fwd_host", lib().tm_trianglemix_attn_fwd_host(
        _ptr(q_host), _ptr(k_host), _ptr(v_host), _ptr(o_host), _ptr(q_dev), _ptr(k_dev),
        _ptr(v_dev), _ptr(o_dev), B, Hq, Hkv, N, D, scale, S, W, L, layer, tri_start,
        int(chunk_rows), _stream(stream)))


def tm_causal_attn_fwd_ws(q, k, v, o, B, Hq, Hkv, N, D, scale, workspace, workspace_bytes,
                          stream=None):
    return _check("tm_causal_attn_fwd_ws", lib().tm_causal_attn_fwd_ws(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), B, Hq, Hkv, N, D, scale, _ptr(workspace),
        int(workspace_bytes), _stream(stream)))


def tm_triangle_attn_fwd_ws(q, k, v, o, B, Hq, Hkv, N, D, scale, S, W, L, workspace,
                            workspace_bytes, stream=None):
    return _check("tm_triangle_attn_fwd_ws", lib().tm_triangle_attn_fwd_ws(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), B, Hq, Hkv, N, D, scale, S, W, L, _ptr(workspace),
        int(workspace_bytes), _stream(stream)))


def tm_trianglemix_attn_fwd_ws(q, k, v, o, B, Hq, Hkv, N, D, scale, S, W, L, layer, tri_start,
                               workspace, workspace_bytes, stream=None):
    return _check("tm_trianglemix_attn_fwd_ws", lib().tm_trianglemix_attn_fwd_ws(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), B, Hq, Hkv, N, D, scale, S, W, L, layer, tri_start,
        _ptr(workspace), int(workspace_bytes), _stream(stream)))


def tm_trianglemix_attn_fwd_noalloc(q, k, v, o, B, Hq, Hkv, N, D, scale, S, W, L, layer,
                                    tri_start, stream=None):
    return _check("tm_trianglemix_attn_fwd_noalloc", lib().tm_trianglemix_attn_fwd_noalloc(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), B, Hq, Hkv, N, D, scale, S, W, L, layer, tri_start,
        _stream(stream)))


TM_NOALLOC_SCRATCH_BYTES = 16 << 20


def tm_block_sparse_attn_fwd(q, k, v, o, B, Hq, Hkv, N, D, scale, block_offsets, block_indices,
                             nnz, stream=None):
    return _check("tm_block_sparse_attn_fwd", lib().tm_block_sparse_attn_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), B, Hq, Hkv, N, D, scale, _ptr(block_offsets),
        _ptr(block_indices), int(nnz), _stream(stream)))


def tm_trianglemix_sparse_attn_fwd(q, k, v, o, B, Hq, Hkv, N, D, scale, S, W, L, layer,
                                   tri_start, block_offsets, block_indices, nnz, stream=None):
    return _check("tm_trianglemix_sparse_attn_fwd", lib().tm_trianglemix_sparse_attn_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), B, Hq, Hkv, N, D, scale, S, W, L, layer, tri_start,
        _ptr(block_offsets), _ptr(block_indices), int(nnz), _stream(stream)))


def tm_triangle_attn_fwd_heads(q, k, v, o, B, Hq, Hkv, N, D, scale, S_heads, W_heads, L,
                               workspace=None, workspace_bytes=0, stream=None):
    """Triangle attention with per-head sinks and windows (host int sequences of Hq)."""
    Sh = np.ascontiguousarray(S_heads, dtype=np.int32)
    Wh = np.ascontiguousarray(W_heads, dtype=np.int32)
    assert Sh.size == Hq and Wh.size == Hq
    return _check("tm_triangle_attn_fwd_heads", lib().tm_triangle_attn_fwd_heads(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), B, Hq, Hkv, N, D, scale, Sh.ctypes.data,
        Wh.ctypes.data, L, _ptr(workspace), int(workspace_bytes), _stream(stream)))


def tm_flashprefill_workspace_size(B, Hq, Hkv, N, D, probes) -> int:
    n = ctypes.c_longlong(0)
    _check("tm_flashprefill_workspace_size", lib().tm_flashprefill_workspace_size(
        B, Hq, Hkv, N, D, probes, ctypes.byref(n)))
    return n.value


def tm_flashprefill_index_capacity(B, Hkv, N) -> int:
    return int(lib().tm_flashprefill_index_capacity(B, Hkv, N))


def tm_flashprefill_block_index(q, k, B, Hq, Hkv, N, D, scale, alpha, probes, workspace,
                                workspace_bytes, block_offsets, block_indices, cap,
                                scores_out=None, stream=None):
    return _check("tm_flashprefill_block_index", lib().tm_flashprefill_block_index(
        _ptr(q), _ptr(k), B, Hq, Hkv, N, D, scale, alpha, probes, _ptr(workspace),
        int(workspace_bytes), _ptr(block_offsets), _ptr(block_indices), int(cap),
        _ptr(scores_out), _stream(stream)))


def tm_attn_workspace_size(B, Hq, Hkv, N, D, causal, S, W, L, num_ctas=0) -> int:
    """Workspace bytes of the split schedule (0: nothing is split)."""
    n = ctypes.c_longlong(0)
    _check("tm_attn_workspace_size", lib().tm_attn_workspace_size(
        B, Hq, Hkv, N, D, int(causal), S, W, L, num_ctas, ctypes.byref(n)))
    return n.value


def tm_triangle_kept_pairs(N, S, W, L) -> int:
    return int(lib().tm_triangle_kept_pairs(N, S, W, L))


def tm_kept_tiles(N, causal, S, W, L) -> int:
    return int(lib().tm_kept_tiles(N, int(causal), S, W, L))


def tm_tile_list(N, causal, S, W, L, BM=TM_BLOCK_M, BN=TM_BLOCK_N) -> np.ndarray:
    """(qb, kb, full) records of the static tile list, as an int32 [n, 3] array."""
    cnt = ctypes.c_longlong(0)
    _check("tm_tile_list", lib().tm_tile_list(N, int(causal), S, W, L, BM, BN, None, 0,
                                              ctypes.byref(cnt)))
    out = np.zeros((max(cnt.value, 1), 3), np.int32)
    _check("tm_tile_list", lib().tm_tile_list(N, int(causal), S, W, L, BM, BN,
                                              out.ctypes.data, cnt.value, ctypes.byref(cnt)))
    return out[: cnt.value]


def tm_triangle_tile_list(N, S, W, L, BM=TM_BLOCK_M, BN=TM_BLOCK_N) -> np.ndarray:
    cnt = ctypes.c_longlong(0)
    _check("tm_triangle_tile_list", lib().tm_triangle_tile_list(N, S, W, L, BM, BN, None, 0,
                                                                ctypes.byref(cnt)))
    out = np.zeros((max(cnt.value, 1), 3), np.int32)
    _check("tm_triangle_tile_list", lib().tm_triangle_tile_list(
        N, S, W, L, BM, BN, out.ctypes.data, cnt.value, ctypes.byref(cnt)))
    return out[: cnt.value]


def tm_debug_dump_tiles(N, causal, S, W, L, out_dev, cap, stream=None) -> int:
    cnt = ctypes.c_longlong(0)
    _check("tm_debug_dump_tiles", lib().tm_debug_dump_tiles(
        N, int(causal), S, W, L, _ptr(out_dev), cap, ctypes.byref(cnt), _stream(stream)))
    return cnt.value


def tm_debug_mma_probe(q, k, v, s_out, o_out, D, stream=None):
    return _check("tm_debug_mma_probe", lib().tm_debug_mma_probe(
        _ptr(q), _ptr(k), _ptr(v), _ptr(s_out), _ptr(o_out), D, _stream(stream)))


def tm_debug_schedule(B, Hq, Hkv, N, causal, S, W, L, num_ctas=148, split=False,
                      mix_pairs=False, qb_lo=0, qb_hi=-1) -> np.ndarray:
    """Persistent work split as an int32 [n, 7] array:
    (cta, item, q-block, head0, Q tiles, first tile, end tile); with a window,
    the split of the q-blocks [qb_lo, qb_hi) only."""
    split = int(bool(split)) | (2 if mix_pairs else 0)
    cnt = ctypes.c_longlong(0)
    f = lib().tm_debug_schedule_window
    _check("tm_debug_schedule_window", f(B, Hq, Hkv, N, int(causal), S, W, L, num_ctas,
                                         int(split), qb_lo, qb_hi, None, 0, ctypes.byref(cnt)))
    out = np.zeros((max(cnt.value, 1), 7), np.int32)
    _check("tm_debug_schedule_window", f(B, Hq, Hkv, N, int(causal), S, W, L, num_ctas,
                                         int(split), qb_lo, qb_hi, out.ctypes.data, cnt.value,
                                         ctypes.byref(cnt)))
    return out[: cnt.value]


def tm_debug_schedule_heads(B, Hq, Hkv, N, S_heads, W_heads, L, num_ctas=148,
                            split=False) -> np.ndarray:
    """tm_debug_schedule of a per-head band launch with these bands (records as there)."""
    hs = np.ascontiguousarray(S_heads, dtype=np.int32)
    hw = np.ascontiguousarray(W_heads, dtype=np.int32)
    cnt = ctypes.c_longlong(0)
    f = lib().tm_debug_schedule_heads
    _check("tm_debug_schedule_heads", f(B, Hq, Hkv, N, hs.ctypes.data, hw.ctypes.data, L, num_ctas,
                                        int(bool(split)), None, 0, ctypes.byref(cnt)))
    out = np.zeros((max(cnt.value, 1), 7), np.int32)
    _check("tm_debug_schedule_heads", f(B, Hq, Hkv, N, hs.ctypes.data, hw.ctypes.data, L, num_ctas,
                                        int(bool(split)), out.ctypes.data, cnt.value,
                                        ctypes.byref(cnt)))
    return out[: cnt.value]


def tm_debug_inject_stall(q, k, v, o, B, Hq, Hkv, N, D, scale, S, W, L, stream=None):
    return _check("tm_debug_inject_stall", lib().tm_debug_inject_stall(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), B, Hq, Hkv, N, D, scale, S, W, L, _stream(stream)))


def _device_ptrs(*xs, strided=0):
    """Addresses of the arguments; a tensor has to lie on the current device (a kernel that
    reads another device's or the host's memory faults), and, but for the first ``strided``
    ones, to be contiguous (the library would read the rows between a slice's)."""
    out, here = [], None
    for x in xs:
        if x is None:
            out.append(None)
            continue
        try:
            device = x.get_device()  # -1: the host
        except AttributeError:
            out.append(operator.index(x))  # an address; not a number that an array holds
            continue
        if device != here:
            if here is not None or device < 0 or device != (_device or _find_current_stream())():
                raise ValueError(f"a tensor on {x.device}, which is not the current CUDA device")
            here = device
        if len(out) >= strided and not x.is_contiguous():
            raise ValueError(f"a tensor of shape {tuple(x.shape)} and strides {x.stride()} is not "
                             "contiguous")
        out.append(x.data_ptr())
    return out


def _rows_apart(x, name, B, N, stride):
    """Elements between consecutive rows of x, whose B sequences of N rows follow each other:
    ``stride``. Where a tensor [B, N, ...] has its rows elsewhere the call is refused, except
    that one row a sequence has no stride of its own (torch may report any): there the stride
    between sequences counts."""
    try:
        own = x.stride()
    except AttributeError:
        return stride  # an address, or nothing
    if N == 1:
        if B == 1 or not own or stride == own[0]:
            return stride
        shape = x.shape
        if len(own) < 3 or shape[0] != B or shape[1] != 1:
            return stride  # a buffer of another shape that the number says how to read
        if stride == own[1]:
            return own[0]
    elif len(own) < 3 or x.size(0) != B or x.size(1) != N or (
            stride == own[1] and (B == 1 or own[0] == N * stride)):
        return stride
    raise ValueError(f"{name}: rows {stride} elements apart do not lie where the strides {own} of "
                     f"its {tuple(x.shape)} put them")


def tm_rope_fwd(q, q_out, k, k_out, B, N, Hq, Hkv, D, q_stride, q_out_stride, k_stride,
                k_out_stride, rot, layout, inverse, inv_freq, mscale, positions, first,
                stream=None):
    q_stride = _rows_apart(q, "q", B, N, q_stride)
    q_out_stride = _rows_apart(q_out, "q_out", B, N, q_out_stride)
    k_stride = _rows_apart(k, "k", B, N, k_stride)
    k_out_stride = _rows_apart(k_out, "k_out", B, N, k_out_stride)
    q, q_out, k, k_out, f, pos = _device_ptrs(q, q_out, k, k_out, inv_freq, positions, strided=4)
    return _check("tm_rope_fwd", lib().tm_rope_fwd(
        q, q_out, k, k_out, B, N, Hq, Hkv, D, q_stride, q_out_stride, k_stride, k_out_stride, rot,
        layout, int(inverse), f, mscale, pos, first, _stream(stream)))


def tm_rope_inv_freq(rot, base, factor=1.0, trained_len=1.0, low_turns=math.inf,
                     high_turns=None) -> np.ndarray:
    """The rotary frequencies (fp64, on the host), stretched by ``factor`` for long contexts: every
    pair, or those of few turns over trained_len where a band of turns is given (high_turns:
    low_turns unless given)."""
    high_turns = low_turns if high_turns is None else high_turns
    out = np.zeros(max(int(rot) // 2, 1), np.float64)
    _check("tm_rope_inv_freq", lib().tm_rope_inv_freq(rot, base, factor, trained_len, low_turns,
                                                      high_turns, out.ctypes.data))
    return out


def tm_kv8_append(k, v, k_stride, v_stride, B, n_src, n, Hkv, D, counts, index, lens, table,
                  max_pages, k8, v8, k_range, v_range, num_pages, page, format, stream=None):
    k_stride = _rows_apart(k, "k", B, n_src, k_stride)
    v_stride = _rows_apart(v, "v", B, n_src, v_stride)
    k, v, counts, index, lens, table, k8, v8, k_range, v_range = _device_ptrs(
        k, v, counts, index, lens, table, k8, v8, k_range, v_range, strided=2)
    return _check("tm_kv8_append", lib().tm_kv8_append(
        k, v, k_stride, v_stride, B, n_src, n, Hkv, D, counts, index, lens, table, max_pages, k8,
        v8, k_range, v_range, num_pages, page, format, _stream(stream)))


def tm_kv8_compact(index, keep, kept, lens, B, Hkv, D, table, max_pages, new_table, new_max_pages,
                   k8, v8, k_range, v_range, num_pages, page, format, weights, weights_stride,
                   new_weights, new_weights_stride, stream=None):
    index, kept, lens, table, new_table, k8, v8, k_range, v_range, weights, new_weights = \
        _device_ptrs(index, kept, lens, table, new_table, k8, v8, k_range, v_range, weights,
                     new_weights)
    return _check("tm_kv8_compact", lib().tm_kv8_compact(
        index, keep, kept, lens, B, Hkv, D, table, max_pages, new_table, new_max_pages, k8, v8,
        k_range, v_range, num_pages, page, format, weights, weights_stride, new_weights,
        new_weights_stride, _stream(stream)))


def tm_kv8_attn_workspace_size(B, nq, Hq, Hkv, D, max_pages, page, with_weights) -> int:
    n = ctypes.c_longlong(0)
    _check("tm_kv8_attn_workspace_size", lib().tm_kv8_attn_workspace_size(
        B, nq, Hq, Hkv, D, max_pages, page, int(bool(with_weights)), ctypes.byref(n)))
    return n.value


def tm_kv8_attn_fwd(q, o, B, nq, Hq, Hkv, D, scale, k8, v8, k_range, v_range, num_pages, page,
                    format, table, max_pages, lens, weights, weights_stride, accumulate,
                    workspace, workspace_bytes, stream=None):
    q, o, k8, v8, k_range, v_range, table, lens, weights, workspace = _device_ptrs(
        q, o, k8, v8, k_range, v_range, table, lens, weights, workspace)
    return _check("tm_kv8_attn_fwd", lib().tm_kv8_attn_fwd(
        q, o, B, nq, Hq, Hkv, D, scale, k8, v8, k_range, v_range, num_pages, page, format, table,
        max_pages, lens, weights, weights_stride, int(accumulate), workspace, workspace_bytes,
        _stream(stream)))


def tm_key_weights_workspace_size(B, Hq, Hkv, N, D, L) -> int:
    n = ctypes.c_longlong(0)
    _check("tm_key_weights_workspace_size", lib().tm_key_weights_workspace_size(
        B, Hq, Hkv, N, D, L, ctypes.byref(n)))
    return n.value


def tm_key_weights_fwd(q, k, B, Hq, Hkv, N, D, scale, L, lens, weights, weights_stride,
                       accumulate, workspace, workspace_bytes, stream=None):
    q, k, lens, weights, workspace = _device_ptrs(q, k, lens, weights, workspace)
    return _check("tm_key_weights_fwd", lib().tm_key_weights_fwd(
        q, k, B, Hq, Hkv, N, D, scale, L, lens, weights, weights_stride, int(accumulate),
        workspace, workspace_bytes, _stream(stream)))


def tm_kv_select(weights, weights_stride, lens, B, H, n, keep, sinks, recent, index, kept=None,
                 stream=None):
    weights, lens, index, kept = _device_ptrs(weights, lens, index, kept)
    return _check("tm_kv_select", lib().tm_kv_select(
        weights, weights_stride, lens, B, H, n, keep, sinks, recent, index, kept,
        _stream(stream)))


def tm_get_device_status(stream=None) -> int:
    return int(lib().tm_get_device_status(_stream(stream)))


def tm_debug_launch_count() -> int:
    return int(lib().tm_debug_launch_count())


# ----------------------------------------------------------------------- torch conveniences

def _shapes(q, k):
    B, N, Hq, D = q.shape
    Hkv = k.shape[2]
    return B, N, Hq, Hkv, D


def _out(q, out):
    import torch
    return torch.empty_like(q) if out is None else out


def causal_attention(q, k, v, scale=None, out=None, stream=None):
    """Dense causal attention of bf16 CUDA tensors q [B,N,Hq,D], k/v [B,N,Hkv,D]."""
    B, N, Hq, Hkv, D = _shapes(q, k)
    o = _out(q, out)
    tm_causal_attn_fwd(q, k, v, o, B, Hq, Hkv, N, D,
                       1.0 / math.sqrt(D) if scale is None else scale, stream)
    return o


def triangle_attention(q, k, v, S, W, L, scale=None, out=None, stream=None):
    """Triangle attention (sinks S, window W, last L rows) of bf16 CUDA tensors."""
    B, N, Hq, Hkv, D = _shapes(q, k)
    o = _out(q, out)
    tm_triangle_attn_fwd(q, k, v, o, B, Hq, Hkv, N, D,
                         1.0 / math.sqrt(D) if scale is None else scale, S, W, L, stream)
    return o


def trianglemix_attention(q, k, v, S, W, L, layer, tri_start, scale=None, out=None, stream=None):
    """One layer of the TriangleMix schedule: causal below tri_start, triangle from it on."""
    B, N, Hq, Hkv, D = _shapes(q, k)
    o = _out(q, out)
    tm_trianglemix_attn_fwd(q, k, v, o, B, Hq, Hkv, N, D,
                            1.0 / math.sqrt(D) if scale is None else scale, S, W, L, layer,
                            tri_start, stream)
    return o


# The operators around the attention, on torch tensors. Token counts and tables are int32 CUDA
# tensors, k and v bf16; shapes and types are checked here, ranges of values on the device. With a
# `stream`, results and workspaces that a call allocates belong to that stream.

def _on(stream):
    """A context in which torch allocates and fills on ``stream`` (None: the current one): a
    workspace given back at the end of a call is then reused behind the call's kernels, and a
    result's zeros are there before them."""
    import torch
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _workspace(workspace, size, device, stream):
    import torch
    if workspace is not None:
        return _need(workspace, "workspace", torch.uint8, None)
    with _on(stream):
        return torch.empty(size, dtype=torch.uint8, device=device)


def _need(x, name, dtype, *shape):
    """x has this dtype and shape (None: any size) and is contiguous."""
    if x.dtype != dtype:
        raise ValueError(f"{name} is {x.dtype}, not {dtype}")
    if x.dim() != len(shape) or any(n is not None and x.shape[i] != n for i, n in enumerate(shape)):
        raise ValueError(f"{name} has shape {tuple(x.shape)}, not {shape}")
    if not x.is_contiguous():
        raise ValueError(f"{name} is not contiguous")
    return x


def _token_rows(x, name, D=None):
    """Token stride of bf16 [B, N, H, D] rows whose heads are contiguous (a slice of a packed
    projection is)."""
    import torch
    if x.dtype != torch.bfloat16 or x.dim() != 4 or (D is not None and x.shape[3] != D):
        raise ValueError(f"{name}: {x.dtype} {tuple(x.shape)} is not bf16 [B, N, H, {D or 'D'}]")
    B, N, H, D = x.shape
    if (D > 1 and x.stride(3) != 1) or (H > 1 and x.stride(2) != D):
        raise ValueError(f"{name}: the heads of a token are not contiguous")
    if N > 1:
        stride = x.stride(1)
        if B > 1 and x.stride(0) != N * stride:
            raise ValueError(f"{name}: the batches do not follow each other")
    else:
        stride = x.stride(0) if B > 1 else H * D
    return stride


def rope(q, k, inv_freq, positions=None, first=0, rot=None, interleaved=False, mscale=1.0,
         inverse=False, out=None, stream=None):
    """Rotary positions of bf16 q [B, N, Hq, D] and k [B, N, Hkv, D] (either may be None, both
    may be slices of a packed projection). ``inv_freq``: rot / 2 doubles on the device
    (tm_rope_inv_freq). ``out``: the pair to write to, (q, k) themselves to turn in place."""
    import torch
    x = q if q is not None else k
    B, N, _, D = x.shape
    rot = D if rot is None else rot
    _need(inv_freq, "inv_freq", torch.float64, rot // 2)
    if positions is not None:
        _need(positions, "positions", torch.int32, B, N)
    if out is None:
        with _on(stream):
            outs = [None if t is None else torch.empty(t.shape, dtype=t.dtype, device=t.device)
                    for t in (q, k)]
    else:
        outs = list(out)
    H, st = [], []
    for t, o, name in ((q, outs[0], "q"), (k, outs[1], "k")):
        if t is None:
            H.append(0)
            st += [0, 0]
            continue
        if t.shape[:2] != (B, N) or t.shape[3] != D or o.shape != t.shape:
            raise ValueError(f"{name}: {tuple(t.shape)} and {tuple(o.shape)} do not fit")
        H.append(t.shape[2])
        st += [_token_rows(t, name), _token_rows(o, name + "'s output")]
    tm_rope_fwd(q, outs[0], k, outs[1], B, N, H[0], H[1], D, *st, rot, int(bool(interleaved)),
                inverse, inv_freq, mscale, positions, first, stream)
    return tuple(outs)


class Kv8Cache(NamedTuple):
    """A paged 8-bit cache: codes [num_pages, Hkv, page, D] (int8 or float8_e4m3fn) and their
    blocks' ranges [num_pages, Hkv]."""
    k8: Any
    v8: Any
    k_range: Any
    v_range: Any

    @staticmethod
    def empty(num_pages, Hkv, page, D, format=TM_KV_INT8, device="cuda"):
        import torch
        dtype = torch.int8 if format == TM_KV_INT8 else torch.float8_e4m3fn
        codes = [torch.zeros((num_pages, Hkv, page, D), dtype=torch.int8, device=device).view(dtype)
                 for _ in range(2)]
        return Kv8Cache(*codes, *(torch.zeros((num_pages, Hkv), device=device) for _ in range(2)))

    def _args(self):
        """(codes and ranges..., num_pages, page, format), checked."""
        import torch
        n, H, page, D = self.k8.shape
        _need(self.k8, "k8", self.k8.dtype, n, H, page, D)
        _need(self.v8, "v8", self.k8.dtype, n, H, page, D)
        _need(self.k_range, "k_range", torch.float32, n, H)
        _need(self.v_range, "v_range", torch.float32, n, H)
        formats = {torch.int8: TM_KV_INT8, torch.float8_e4m3fn: TM_KV_E4M3}
        if self.k8.dtype not in formats:
            raise ValueError(f"codes of {self.k8.dtype}")
        return (self.k8, self.v8, self.k_range, self.v_range, n, page, formats[self.k8.dtype])


def kv8_append(cache, k, v, lens, table, counts=None, index=None, stream=None):
    """Store bf16 k, v [B, n, Hkv, D] behind the lens[b] tokens a sequence holds (lens is not
    changed); only the first counts[b], or the rows index [B, Hkv, n] of each head."""
    import torch
    _, H, _, D = cache.k8.shape
    B, n_src = k.shape[:2]
    ks, vs = _token_rows(k, "k", D), _token_rows(v, "v", D)
    if v.shape != k.shape or k.shape[2] != H:
        raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)} for {H} heads")
    n = n_src
    if index is not None:
        n = _need(index, "index", torch.int32, B, H, None).shape[2]
    if counts is not None:
        _need(counts, "counts", torch.int32, B)
    _need(lens, "lens", torch.int32, B)
    _need(table, "table", torch.int32, B, None)
    tm_kv8_append(k, v, ks, vs, B, n_src, n, H, D, counts, index, lens, table, table.shape[1],
                  *cache._args(), stream)


def kv8_attention(cache, q, lens, table, scale=None, weights=None, accumulate=False, out=None,
                  workspace=None, stream=None):
    """Attention of the last nq tokens, bf16 q [B, nq, Hq, D], over the cache; the weight of each
    key into ``weights`` [B, Hkv, tokens] if given. A ``workspace`` (uint8) saves its allocation."""
    import torch
    B, nq, Hq, D = q.shape
    _, H, page, Dc = cache.k8.shape
    _need(q, "q", torch.bfloat16, B, nq, Hq, Dc)
    _need(lens, "lens", torch.int32, B)
    mp = _need(table, "table", torch.int32, B, None).shape[1]
    if weights is not None:
        _need(weights, "weights", torch.float32, B, H, None)
    with _on(stream):
        o = _out(q, out)
    _need(o, "out", torch.bfloat16, B, nq, Hq, D)
    size = tm_kv8_attn_workspace_size(B, nq, Hq, H, D, mp, page, weights is not None)
    workspace = _workspace(workspace, size, q.device, stream)
    tm_kv8_attn_fwd(q, o, B, nq, Hq, H, D, 1.0 / math.sqrt(D) if scale is None else scale,
                    *cache._args(), table, mp, lens, weights,
                    0 if weights is None else weights.shape[2], accumulate, workspace,
                    workspace.numel(), stream)
    return o


def key_weights(q, k, L, lens=None, scale=None, weights=None, accumulate=False, workspace=None,
                stream=None):
    """The attention weight each key of bf16 k [B, N, Hkv, D] receives from the last L queries of
    q [B, N, Hq, D], [B, Hkv, N] (keys past a sequence's length stay as they are, 0 if new)."""
    import torch
    B, N, Hq, Hkv, D = _shapes(q, k)
    _need(q, "q", torch.bfloat16, B, N, Hq, D)
    _need(k, "k", torch.bfloat16, B, N, Hkv, D)
    if lens is not None:
        _need(lens, "lens", torch.int32, B)
    if weights is None:
        with _on(stream):
            weights = torch.zeros((B, Hkv, N), device=q.device)
    _need(weights, "weights", torch.float32, B, Hkv, None)
    size = tm_key_weights_workspace_size(B, Hq, Hkv, N, D, L)
    workspace = _workspace(workspace, size, q.device, stream)
    tm_key_weights_fwd(q, k, B, Hq, Hkv, N, D, 1.0 / math.sqrt(D) if scale is None else scale, L,
                       lens, weights, weights.shape[2], accumulate, workspace,
                       workspace.numel(), stream)
    return weights


def kv_select(weights, keep, sinks=0, recent=0, lens=None, n=None, stream=None):
    """(index [B, H, keep], kept [B]): the tokens to keep of weights [B, H, tokens], of which the
    first n (all) or lens[b] are there."""
    import torch
    B, H, cap = _need(weights, "weights", torch.float32, None, None, None).shape
    if lens is not None:
        _need(lens, "lens", torch.int32, B)
    with _on(stream):
        index = torch.empty((B, H, keep), dtype=torch.int32, device=weights.device)
        kept = torch.empty(B, dtype=torch.int32, device=weights.device)
    tm_kv_select(weights, cap, lens, B, H, cap if n is None else n, keep, sinks, recent, index, kept,
                 stream)
    return index, kept


def kv8_compact(cache, index, kept, lens, table, new_table, weights=None, new_weights=None,
                stream=None):
    """Move the kept tokens (index [B, Hkv, keep], kept [B]) from table's pages to new_table's,
    and their weights along."""
    import torch
    _, H, _, D = cache.k8.shape
    B, _, keep = _need(index, "index", torch.int32, None, H, None).shape
    _need(kept, "kept", torch.int32, B)
    _need(lens, "lens", torch.int32, B)
    _need(table, "table", torch.int32, B, None)
    _need(new_table, "new_table", torch.int32, B, None)
    for w, name in ((weights, "weights"), (new_weights, "new_weights")):
        if w is not None:
            _need(w, name, torch.float32, B, H, None)
    tm_kv8_compact(index, keep, kept, lens, B, H, D, table, table.shape[1], new_table,
                   new_table.shape[1], *cache._args(), weights,
                   0 if weights is None else weights.shape[2], new_weights,
                   0 if new_weights is None else new_weights.shape[2], stream)
