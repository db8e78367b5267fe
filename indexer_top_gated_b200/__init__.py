"""Python binding of libdsa.so, the B200 gated Indexer + Top-K sparse-attention layer.

Argument marshalling only: every step of the layer runs in the library's CUDA kernels.
Functions carry the C names (``dsa_index_scores``, ``dsa_topk``,
``dsa_sparse_attn_gated``, ``dsa_prefill``, ``dsa_decode``, ...) and take torch CUDA
tensors, which supply device memory and the current stream.  There is no fallback:
if the library cannot be loaded, importing this module raises.
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass
from typing import Optional, Sequence

from . import _build

DSA_OK, DSA_ERR_INVALID_ARG, DSA_ERR_UNSUPPORTED, DSA_ERR_WORKSPACE, DSA_ERR_CUDA, \
    DSA_ERR_TIMEOUT = range(6)
DSA_BF16, DSA_FP8_E4M3 = 0, 1
DSA_ROPE_HALF, DSA_ROPE_INTERLEAVED = 0, 1
DSA_ROPE_SCALE_NONE, DSA_ROPE_SCALE_LINEAR, DSA_ROPE_SCALE_NTK, DSA_ROPE_SCALE_BY_PARTS = range(4)

LIB_PATH = _build.LIB


class DsaError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)} ({status})")
        self.status = status


class Params(ctypes.Structure):
    _fields_ = [
        ("n_idx_heads", ctypes.c_int32), ("idx_dim", ctypes.c_int32),
        ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("top_k", ctypes.c_int32),
        ("idx_dtype", ctypes.c_int32), ("idx_scale_q", ctypes.c_float),
        ("idx_scale_k", ctypes.c_float), ("attn_scale", ctypes.c_float),
        ("w_row_stride", ctypes.c_int32),
    ]


class Ragged(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("q_offsets", ctypes.c_void_p),
        ("kv_offsets", ctypes.c_void_p), ("max_q_len", ctypes.c_int32),
        ("max_kv_len", ctypes.c_int32), ("total_q", ctypes.c_int64),
        ("total_kv", ctypes.c_int64), ("block_table", ctypes.c_void_p),
        ("max_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("q_offsets_host", ctypes.c_void_p), ("kv_offsets_host", ctypes.c_void_p),
    ]


class LayerBuffers(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "q_offsets", "kv_offsets", "q_idx", "k_idx", "w", "q", "k_cache", "v_cache", "gate", "out")]


LAYER_BUFFER_KEYS = ("q_offsets", "kv_offsets", "q_idx", "k_idx", "w", "q", "k", "v", "gate", "out")


def layer_buffers(t: dict) -> LayerBuffers:
    """dsa_layer_buffers from a dict of tensors keyed q_offsets, kv_offsets, q_idx, k_idx, w,
    q, k, v, gate (optional), out."""
    return LayerBuffers(*[_ptr(t.get(k)) for k in LAYER_BUFFER_KEYS])


class RopeParams(ctypes.Structure):
    _fields_ = [
        ("layout", ctypes.c_int32), ("scaling", ctypes.c_int32),
        ("rot_dim", ctypes.c_int32), ("rot_offset", ctypes.c_int32),
        ("idx_rot_dim", ctypes.c_int32), ("idx_rot_offset", ctypes.c_int32),
        ("theta", ctypes.c_double), ("factor", ctypes.c_double), ("orig_len", ctypes.c_double),
        ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double),
        ("magnitude", ctypes.c_double),
        ("q_row_stride", ctypes.c_int64), ("k_row_stride", ctypes.c_int64),
        ("v_row_stride", ctypes.c_int64), ("q_idx_row_stride", ctypes.c_int64),
        ("k_idx_row_stride", ctypes.c_int64),
    ]


class RopeBuffers(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "q", "k", "v", "q_idx", "k_idx", "q_out", "k_cache", "v_cache", "q_idx_out",
        "k_idx_cache")]


class ConvParams(ctypes.Structure):
    _fields_ = [
        ("channels", ctypes.c_int32), ("width", ctypes.c_int32), ("silu", ctypes.c_int32),
        ("n_states", ctypes.c_int32), ("x_row_stride", ctypes.c_int64),
        ("out_row_stride", ctypes.c_int64),
    ]


class DeltaParams(ctypes.Structure):
    _fields_ = [
        ("n_k_heads", ctypes.c_int32), ("n_v_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("qk_norm", ctypes.c_int32),
        ("norm_eps", ctypes.c_float), ("scale", ctypes.c_float),
        ("n_states", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("q_row_stride", ctypes.c_int64), ("k_row_stride", ctypes.c_int64),
        ("v_row_stride", ctypes.c_int64),
    ]


EXPORTS = [
    "dsa_status_string", "dsa_version", "dsa_index_scores", "dsa_topk",
    "dsa_sparse_attn_gated", "dsa_workspace_size", "dsa_prefill", "dsa_decode",
    "dsa_device_status", "dsa_launch_count", "dsa_stage_timing", "dsa_stage_times",
    "dsa_decode_noalloc", "dsa_index_topk", "dsa_index_topk_workspace_size",
    "dsa_sparse_attn_gated_mix", "dsa_index_topk_blocks", "dsa_index_topk_blocks_workspace_size",
    "dsa_prefill_from_host", "dsa_fused_rows", "dsa_rope_append", "dsa_short_conv",
    "dsa_gated_delta_workspace_size", "dsa_gated_delta_prefill", "dsa_gated_delta_decode",
]


def _load():
    _build.build()
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    PP, RP = ctypes.POINTER(Params), ctypes.POINTER(Ragged)
    L.dsa_status_string.argtypes = [ctypes.c_int]
    L.dsa_status_string.restype = ctypes.c_char_p
    L.dsa_version.argtypes = []
    L.dsa_version.restype = i32
    L.dsa_index_scores.argtypes = [PP, RP, vp, vp, vp, i64, i64, vp, i64, vp]
    L.dsa_topk.argtypes = [PP, RP, vp, i64, i64, i64, vp, i64, vp, vp]
    L.dsa_sparse_attn_gated.argtypes = [PP, RP, vp, vp, vp, vp, i64, i64, i64, vp, vp, vp, vp, vp]
    LB = ctypes.POINTER(LayerBuffers)
    L.dsa_prefill_from_host.argtypes = [PP, RP, LB, LB, i32, i32, vp, sz, vp]
    L.dsa_index_topk_blocks_workspace_size.argtypes = [PP, RP, i32, i64, ctypes.POINTER(sz),
                                                       ctypes.POINTER(sz)]
    L.dsa_index_topk_blocks.argtypes = [PP, RP, vp, vp, vp, i32, i64, i64, vp, i64, vp, vp, sz, vp]
    L.dsa_sparse_attn_gated_mix.argtypes = [PP, RP, vp, vp, vp, vp, i64, i64, i64, vp, vp, vp, vp,
                                            vp, vp]
    L.dsa_workspace_size.argtypes = [PP, RP, ctypes.c_int, ctypes.POINTER(sz), ctypes.POINTER(sz)]
    L.dsa_index_topk_workspace_size.argtypes = [PP, RP, i64, ctypes.POINTER(sz), ctypes.POINTER(sz)]
    L.dsa_index_topk.argtypes = [PP, RP, vp, vp, vp, i64, i64, vp, i64, vp, vp, sz, vp]
    L.dsa_prefill.argtypes = [PP, RP, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.dsa_decode.argtypes = L.dsa_prefill.argtypes
    L.dsa_decode_noalloc.argtypes = [PP, RP, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.dsa_device_status.argtypes = [vp, ctypes.POINTER(i32), ctypes.c_int]
    L.dsa_launch_count.argtypes = []
    L.dsa_launch_count.restype = i64
    L.dsa_fused_rows.argtypes = [ctypes.c_int]
    L.dsa_fused_rows.restype = i64
    L.dsa_stage_timing.argtypes = [ctypes.c_int]
    L.dsa_stage_times.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(i64), ctypes.c_int]
    L.dsa_rope_append.argtypes = [PP, RP, ctypes.POINTER(RopeParams), ctypes.POINTER(RopeBuffers),
                                  vp, vp, vp]
    L.dsa_short_conv.argtypes = [ctypes.POINTER(ConvParams), RP, vp, vp, vp, vp, vp, vp, vp, vp]
    DP = ctypes.POINTER(DeltaParams)
    L.dsa_gated_delta_workspace_size.argtypes = [DP, RP, ctypes.POINTER(sz), ctypes.POINTER(sz)]
    L.dsa_gated_delta_prefill.argtypes = [DP, RP, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.dsa_gated_delta_decode.argtypes = [DP, RP, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    for name in ("dsa_index_scores", "dsa_topk", "dsa_sparse_attn_gated", "dsa_workspace_size",
                 "dsa_prefill", "dsa_decode", "dsa_decode_noalloc", "dsa_device_status",
                 "dsa_stage_timing",
                 "dsa_stage_times"):
        getattr(L, name).restype = ctypes.c_int
    return L


lib = _load()


def status_string(s: int) -> str:
    return lib.dsa_status_string(int(s)).decode()


def _check(rc: int, where: str):
    if rc != DSA_OK:
        raise DsaError(rc, where)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream) -> int:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


@dataclass
class LayerShape:
    n_idx_heads: int = 4
    idx_dim: int = 64
    n_q_heads: int = 32
    n_kv_heads: int = 4
    head_dim: int = 128
    top_k: int = 2048
    idx_dtype: int = DSA_BF16
    idx_scale_q: float = 1.0
    idx_scale_k: float = 1.0
    attn_scale: float = 0.0
    w_row_stride: int = 0

    def params(self) -> Params:
        return Params(self.n_idx_heads, self.idx_dim, self.n_q_heads, self.n_kv_heads,
                      self.head_dim, self.top_k, self.idx_dtype, self.idx_scale_q,
                      self.idx_scale_k, self.attn_scale, self.w_row_stride)


def ragged(q_offsets, kv_offsets, q_lens: Sequence[int], kv_lens: Sequence[int],
           block_table=None, page_size: int = 0, cache_rows: Optional[int] = None) -> Ragged:
    """Build a dsa_ragged from device int32 offset tensors and host lengths; with a device
    int32 block table [batch, max_pages] the cache arrays are paged (cache_rows rows).
    Host copies of the offsets are made from the lengths and attached (they let the layer
    plan per sequence).  The descriptor holds only the tensors' addresses: keep them alive
    while it is used."""
    import numpy as np
    qoh = np.concatenate([[0], np.cumsum(np.asarray(q_lens, dtype=np.int64))]).astype(np.int32)
    koh = np.concatenate([[0], np.cumsum(np.asarray(kv_lens, dtype=np.int64))]).astype(np.int32)
    rg = Ragged(len(q_lens), q_offsets.data_ptr(), kv_offsets.data_ptr(),
                int(max(q_lens)) if len(q_lens) else 0,
                int(max(kv_lens)) if len(kv_lens) else 0, int(sum(q_lens)), int(sum(kv_lens)),
                None, 0, 0, qoh.ctypes.data, koh.ctypes.data)
    rg.host_offsets = (qoh, koh)  # keeps the host copies alive with the descriptor
    if block_table is not None:
        rg.block_table = block_table.data_ptr()
        rg.max_pages = int(block_table.shape[1])
        rg.page_size = int(page_size)
        rg.total_kv = int(cache_rows)
    return rg


def dsa_index_scores(shape: LayerShape, rg: Ragged, q_idx, k_idx, w, q_begin: int, q_count: int,
                     scores, ld_scores: int, stream=None):
    p = shape.params()
    _check(lib.dsa_index_scores(ctypes.byref(p), ctypes.byref(rg), _ptr(q_idx), _ptr(k_idx),
                                _ptr(w), q_begin, q_count, _ptr(scores), ld_scores,
                                _stream(stream)), "dsa_index_scores")


def dsa_topk(shape: LayerShape, rg: Ragged, scores, ld_scores: int, q_begin: int, q_count: int,
             idx, ld_idx: int, cnt=None, stream=None):
    p = shape.params()
    _check(lib.dsa_topk(ctypes.byref(p), ctypes.byref(rg), _ptr(scores), ld_scores, q_begin,
                        q_count, _ptr(idx), ld_idx, _ptr(cnt), _stream(stream)), "dsa_topk")


def dsa_sparse_attn_gated(shape: LayerShape, rg: Ragged, q, k_cache, v_cache, idx, ld_idx: int,
                          q_begin: int, q_count: int, gate, out, lse=None, err_count=None,
                          stream=None):
    p = shape.params()
    _check(lib.dsa_sparse_attn_gated(ctypes.byref(p), ctypes.byref(rg), _ptr(q), _ptr(k_cache),
                                     _ptr(v_cache), _ptr(idx), ld_idx, q_begin, q_count,
                                     _ptr(gate), _ptr(out), _ptr(lse), _ptr(err_count),
                                     _stream(stream)), "dsa_sparse_attn_gated")


def dsa_prefill_from_host(shape: LayerShape, rg: Ragged, host: dict, dev: dict, n_chunks: int = 0,
                          workspace=None, ws_bytes=None, stream=None, order: int = 0):
    """dsa_prefill with inputs and output in (page-locked) host tensors, copies overlapped
    with the computation; dev holds the device buffers of the same shapes."""
    p = shape.params()
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size()
    hb, db = layer_buffers(host), layer_buffers(dev)
    _check(lib.dsa_prefill_from_host(ctypes.byref(p), ctypes.byref(rg), ctypes.byref(hb),
                                     ctypes.byref(db), n_chunks, order, _ptr(workspace), ws_bytes,
                                     _stream(stream)), "dsa_prefill_from_host")


def dsa_index_topk_blocks_workspace_size(shape: LayerShape, rg: Ragged, block: int,
                                         q_count: int):
    p = shape.params()
    mn, rec = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib.dsa_index_topk_blocks_workspace_size(ctypes.byref(p), ctypes.byref(rg), block,
                                                    q_count, ctypes.byref(mn), ctypes.byref(rec)),
           "dsa_index_topk_blocks_workspace_size")
    return mn.value, rec.value


def dsa_index_topk_blocks(shape: LayerShape, rg: Ragged, q_idx, k_idx, w, block: int, q_begin: int,
                          q_count: int, idx, ld_idx: int, cnt=None, workspace=None, ws_bytes=None,
                          stream=None):
    """top_k of `shape` counts blocks; idx receives positions (ld_idx >= top_k * block)."""
    p = shape.params()
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.dsa_index_topk_blocks(ctypes.byref(p), ctypes.byref(rg), _ptr(q_idx), _ptr(k_idx),
                                     _ptr(w), block, q_begin, q_count, _ptr(idx), ld_idx,
                                     _ptr(cnt), _ptr(workspace), ws_bytes, _stream(stream)),
           "dsa_index_topk_blocks")


def dsa_sparse_attn_gated_mix(shape: LayerShape, rg: Ragged, q, k_cache, v_cache, idx, ld_idx: int,
                              q_begin: int, q_count: int, gate, other, out, lse=None,
                              err_count=None, stream=None):
    p = shape.params()
    _check(lib.dsa_sparse_attn_gated_mix(ctypes.byref(p), ctypes.byref(rg), _ptr(q),
                                         _ptr(k_cache), _ptr(v_cache), _ptr(idx), ld_idx, q_begin,
                                         q_count, _ptr(gate), _ptr(other), _ptr(out), _ptr(lse),
                                         _ptr(err_count), _stream(stream)),
           "dsa_sparse_attn_gated_mix")


def dsa_workspace_size(shape: LayerShape, rg: Ragged, is_decode: bool = False):
    p = shape.params()
    mn, rec = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib.dsa_workspace_size(ctypes.byref(p), ctypes.byref(rg), int(is_decode),
                                  ctypes.byref(mn), ctypes.byref(rec)), "dsa_workspace_size")
    return mn.value, rec.value


def dsa_index_topk_workspace_size(shape: LayerShape, rg: Ragged, q_count: int):
    p = shape.params()
    mn, rec = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib.dsa_index_topk_workspace_size(ctypes.byref(p), ctypes.byref(rg), q_count,
                                             ctypes.byref(mn), ctypes.byref(rec)),
           "dsa_index_topk_workspace_size")
    return mn.value, rec.value


def dsa_index_topk(shape: LayerShape, rg: Ragged, q_idx, k_idx, w, q_begin: int, q_count: int,
                   idx, ld_idx: int, cnt=None, workspace=None, ws_bytes=None, stream=None):
    p = shape.params()
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.dsa_index_topk(ctypes.byref(p), ctypes.byref(rg), _ptr(q_idx), _ptr(k_idx),
                              _ptr(w), q_begin, q_count, _ptr(idx), ld_idx, _ptr(cnt),
                              _ptr(workspace), ws_bytes, _stream(stream)), "dsa_index_topk")


def _layer(fn, name, shape, rg, q_idx, k_idx, w, q, k_cache, v_cache, gate, out, idx_out,
           err_count, workspace, ws_bytes, stream):
    p = shape.params()
    if ws_bytes is None:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check(fn(ctypes.byref(p), ctypes.byref(rg), _ptr(q_idx), _ptr(k_idx), _ptr(w), _ptr(q),
              _ptr(k_cache), _ptr(v_cache), _ptr(gate), _ptr(out), _ptr(idx_out), _ptr(err_count),
              _ptr(workspace), ws_bytes, _stream(stream)), name)


def dsa_prefill(shape: LayerShape, rg: Ragged, q_idx, k_idx, w, q, k_cache, v_cache, gate, out,
                idx_out=None, err_count=None, workspace=None, ws_bytes=None, stream=None):
    _layer(lib.dsa_prefill, "dsa_prefill", shape, rg, q_idx, k_idx, w, q, k_cache, v_cache, gate,
           out, idx_out, err_count, workspace, ws_bytes, stream)


def dsa_decode(shape: LayerShape, rg: Ragged, q_idx, k_idx, w, q, k_cache, v_cache, gate, out,
               idx_out=None, err_count=None, workspace=None, ws_bytes=None, stream=None):
    _layer(lib.dsa_decode, "dsa_decode", shape, rg, q_idx, k_idx, w, q, k_cache, v_cache, gate,
           out, idx_out, err_count, workspace, ws_bytes, stream)


def dsa_decode_noalloc(shape: LayerShape, rg: Ragged, q_idx, k_idx, w, q, k_cache, v_cache, gate,
                       out, idx_out=None, err_count=None, stream=None):
    """dsa_decode whose scratch is the library's fixed per-device array (no allocation)."""
    p = shape.params()
    _check(lib.dsa_decode_noalloc(ctypes.byref(p), ctypes.byref(rg), _ptr(q_idx), _ptr(k_idx),
                                  _ptr(w), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(gate),
                                  _ptr(out), _ptr(idx_out), _ptr(err_count), _stream(stream)),
           "dsa_decode_noalloc")


# ---------------------------------------------------------------- around the layer
#
# These take torch tensors whose rows may be slices of wider ones (a fused projection's output):
# row strides come from the tensors, and types, sizes and the device are checked here, since the
# library sees addresses only.

@dataclass(frozen=True)
class RopeShape:
    """Rotary layout, the rotated part of a head, and its frequencies (dsa_rope_params)."""
    layout: int = DSA_ROPE_HALF
    rot_dim: int = 128
    idx_rot_dim: int = 64
    rot_offset: int = 0
    idx_rot_offset: int = 0
    scaling: int = DSA_ROPE_SCALE_NONE
    theta: float = 10000.0
    factor: float = 1.0
    orig_len: float = 4096.0
    beta_fast: float = 32.0
    beta_slow: float = 1.0
    magnitude: float = 1.0

    def __post_init__(self):
        object.__setattr__(self, "_params", RopeParams(
            self.layout, self.scaling, self.rot_dim, self.rot_offset, self.idx_rot_dim,
            self.idx_rot_offset, self.theta, self.factor, self.orig_len, self.beta_fast,
            self.beta_slow, self.magnitude))

    def params(self) -> RopeParams:
        return RopeParams.from_buffer_copy(self._params)


@dataclass(frozen=True)
class ConvShape:
    """Channels, taps and activation of the short convolution (dsa_conv_params)."""
    channels: int
    width: int = 4
    silu: bool = True


@dataclass(frozen=True)
class DeltaShape:
    """Heads and numerics of the gated delta rule (dsa_delta_params)."""
    n_k_heads: int
    n_v_heads: int
    head_dim: int = 128
    qk_norm: bool = True
    norm_eps: float = 1e-6
    scale: float = 0.0


def _bad(where: str, what: str):
    raise DsaError(DSA_ERR_INVALID_ARG, f"{where}: {what}")


def _tensor(where, name, t, dtype, shape, device) -> int:
    """Address of a dense tensor of at least shape[0] rows and exactly the other sizes."""
    if t.dtype is not dtype or t.get_device() != device:
        _bad(where, f"{name} is {t.dtype} on {t.device}, not {dtype} on cuda:{device}")
    if t.shape != shape and (t.dim() != len(shape) or t.shape[0] < shape[0]
                             or t.shape[1:] != shape[1:]):
        _bad(where, f"{name} has shape {tuple(t.shape)}, not {shape}")
    if not t.is_contiguous():
        _bad(where, f"{name} is not contiguous")
    return t.data_ptr()


def _rows(where, name, t, dtype, shape, device):
    """Address and row stride (0: packed) of a tensor whose rows are dense."""
    if t.is_contiguous():
        return _tensor(where, name, t, dtype, shape, device), 0
    if t.dtype is not dtype or t.get_device() != device:
        _bad(where, f"{name} is {t.dtype} on {t.device}, not {dtype} on cuda:{device}")
    if t.shape != shape and (t.dim() != len(shape) or t.shape[0] < shape[0]
                             or t.shape[1:] != shape[1:]):
        _bad(where, f"{name} has shape {tuple(t.shape)}, not {shape}")
    steps, dense = t.stride(), 1
    for i in range(len(shape) - 1, 0, -1):
        if steps[i] != dense and shape[i] > 1:
            _bad(where, f"{name} has rows that are not dense (strides {steps})")
        dense *= shape[i]
    if shape[0] > 1 and steps[0] < dense:  # repeated or overlapping (0 would mean packed)
        _bad(where, f"{name} has rows that are not apart (strides {steps})")
    return t.data_ptr(), steps[0]


def _torch():
    """torch, imported on first use (loading the library does not need it)."""
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


_torch_module = None


def _device(stream) -> int:
    device = _torch().cuda.current_device()
    if stream is not None and stream.device.index != device:
        _bad("stream", f"of {stream.device} while cuda:{device} is current")
    return device


def _raw_stream(stream, device) -> int:
    """Handle of `stream`, or of the device's current one (without building a Stream object)."""
    return _torch()._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


def _output(where, name, t, dtype, shape, device) -> int:
    if t is None:
        _bad(where, f"an input without its {name}")
    return _tensor(where, name, t, dtype, shape, device)


def _index(where, name, t, n, device):
    return None if t is None else _tensor(where, name, t, _torch().int32, (n,), device)


def dsa_rope_append(shape: LayerShape, rg: Ragged, rope: RopeShape, q=None, k=None, v=None,
                    q_idx=None, k_idx=None, q_out=None, k_cache=None, v_cache=None,
                    q_idx_out=None, k_idx_cache=None, positions=None, err_count=None, stream=None):
    """Rotary positions of the batch's new rows: q and q_idx to q_out and q_idx_out, k, v and
    k_idx to the cache rows of their positions.  Inputs left out leave their outputs out."""
    where, device, torch = "dsa_rope_append", _device(stream), _torch()
    bf16 = torch.bfloat16
    idx_type = torch.float8_e4m3fn if shape.idx_dtype == DSA_FP8_E4M3 else bf16
    o, b = rope.params(), RopeBuffers()
    n, rows, d, di = rg.total_q, rg.total_kv, shape.head_dim, shape.idx_dim

    if q is not None:
        shp = (n, shape.n_q_heads, d)
        b.q, o.q_row_stride = _rows(where, "q", q, bf16, shp, device)
        b.q_out = _output(where, "q_out", q_out, bf16, shp, device)
    if k is not None:
        b.k, o.k_row_stride = _rows(where, "k", k, bf16, (n, shape.n_kv_heads, d), device)
        b.k_cache = _output(where, "k_cache", k_cache, bf16, (rows, shape.n_kv_heads, d), device)
    if v is not None:
        b.v, o.v_row_stride = _rows(where, "v", v, bf16, (n, shape.n_kv_heads, d), device)
        b.v_cache = _output(where, "v_cache", v_cache, bf16, (rows, shape.n_kv_heads, d), device)
    if q_idx is not None:
        shp = (n, shape.n_idx_heads, di)
        b.q_idx, o.q_idx_row_stride = _rows(where, "q_idx", q_idx, bf16, shp, device)
        b.q_idx_out = _output(where, "q_idx_out", q_idx_out, idx_type, shp, device)
    if k_idx is not None:
        ni = shape.n_idx_heads
        b.k_idx, o.k_idx_row_stride = _rows(where, "k_idx", k_idx, bf16, (n, ni, di), device)
        b.k_idx_cache = _output(where, "k_idx_cache", k_idx_cache, idx_type, (rows, ni, di), device)
    rc = lib.dsa_rope_append(ctypes.byref(shape.params()), ctypes.byref(rg), ctypes.byref(o),
                             ctypes.byref(b), _index(where, "positions", positions, n, device),
                             _index(where, "err_count", err_count, 1, device),
                             _raw_stream(stream, device))
    _check(rc, where)


def dsa_short_conv(conv: ConvShape, rg: Ragged, x, weight, out, bias=None, state_in=None,
                   state_out=None, state_index=None, stream=None):
    """Short causal convolution of x [total_q, channels] into out, rows before a sequence's
    first from state_in [slots, width - 1, channels], the last ones to state_out."""
    where, device = "dsa_short_conv", _device(stream)
    bf16, c = _torch().bfloat16, conv.channels
    px, sx = _rows(where, "x", x, bf16, (rg.total_q, c), device)
    po, so = _rows(where, "out", out, bf16, (rg.total_q, c), device)
    pw = _tensor(where, "weight", weight, bf16, (c, conv.width), device)
    pb = None if bias is None else _tensor(where, "bias", bias, bf16, (c,), device)
    n, s0, s1 = _states(where, state_in, state_out, bf16, (conv.width - 1, c), device)
    p = ConvParams(c, conv.width, int(conv.silu), n, sx, so)
    _check(lib.dsa_short_conv(ctypes.byref(p), ctypes.byref(rg), px, pw, pb, s0, s1,
                              _index(where, "state_index", state_index, rg.batch, device), po,
                              _raw_stream(stream, device)), where)


def _states(where, state_in, state_out, dtype, slot, device):
    """Slots and addresses of the states before and after (either may be None)."""
    n = 0 if state_in is None and state_out is None else \
        min(t.shape[0] for t in (state_in, state_out) if t is not None)
    shape = (n, *slot)
    return n, None if state_in is None else _tensor(where, "state_in", state_in, dtype, shape, device), \
        None if state_out is None else _tensor(where, "state_out", state_out, dtype, shape, device)


def _delta_params(delta: DeltaShape, n_states: int = 0, strides=(0, 0, 0)) -> DeltaParams:
    return DeltaParams(delta.n_k_heads, delta.n_v_heads, delta.head_dim, int(delta.qk_norm),
                       delta.norm_eps, delta.scale, n_states, 0, *strides)


def _delta_args(where, delta, rg, q, k, v, g, beta, out, state_in, state_out, state_index, device):
    bf16, f32 = _torch().bfloat16, _torch().float32
    n, hv, d = rg.total_q, delta.n_v_heads, delta.head_dim
    qk, vo, gb = (n, delta.n_k_heads, d), (n, hv, d), (n, hv)
    pq, sq = _rows(where, "q", q, bf16, qk, device)
    pk, sk = _rows(where, "k", k, bf16, qk, device)
    pv, sv = _rows(where, "v", v, bf16, vo, device)
    pg = _tensor(where, "g", g, f32, gb, device)
    pb = _tensor(where, "beta", beta, f32, gb, device)
    po = _tensor(where, "out", out, bf16, vo, device)
    ns, s0, s1 = _states(where, state_in, state_out, f32, (hv, d, d), device)
    pi = _index(where, "state_index", state_index, rg.batch, device)
    return _delta_params(delta, ns, (sq, sk, sv)), (pq, pk, pv, pg, pb, s0, s1, pi, po)


def _workspace(where, workspace, ws_bytes, device):
    """Address and bytes of a workspace tensor (ws_bytes of it, or all)."""
    if workspace is None:
        return None, 0
    if workspace.get_device() != device:
        _bad(where, f"workspace on {workspace.device}, not cuda:{device}")
    if not workspace.is_contiguous():
        _bad(where, "workspace is not contiguous")
    held = workspace.numel() * workspace.element_size()
    if ws_bytes is not None and not 0 <= ws_bytes <= held:
        _bad(where, f"ws_bytes is {ws_bytes}, the workspace has {held}")
    return workspace.data_ptr(), held if ws_bytes is None else ws_bytes


def dsa_gated_delta_workspace_size(delta: DeltaShape, rg: Ragged):
    p = _delta_params(delta)
    mn, rec = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib.dsa_gated_delta_workspace_size(ctypes.byref(p), ctypes.byref(rg), ctypes.byref(mn),
                                              ctypes.byref(rec)), "dsa_gated_delta_workspace_size")
    return mn.value, rec.value


def dsa_gated_delta_prefill(delta: DeltaShape, rg: Ragged, q, k, v, g, beta, out, state_in=None,
                            state_out=None, state_index=None, workspace=None, ws_bytes=None,
                            stream=None):
    """The gated delta rule over a ragged batch: out [total_q, Hv, d], states [slots, Hv, dv, dk]."""
    where, device = "dsa_gated_delta_prefill", _device(stream)
    p, args = _delta_args(where, delta, rg, q, k, v, g, beta, out, state_in, state_out,
                          state_index, device)
    _check(lib.dsa_gated_delta_prefill(ctypes.byref(p), ctypes.byref(rg), *args,
                                       *_workspace(where, workspace, ws_bytes, device),
                                       _raw_stream(stream, device)), where)


def dsa_gated_delta_decode(delta: DeltaShape, rg: Ragged, q, k, v, g, beta, out, state_in=None,
                           state_out=None, state_index=None, stream=None):
    """dsa_gated_delta_prefill for at most one token per sequence, without a workspace."""
    where, device = "dsa_gated_delta_decode", _device(stream)
    p, args = _delta_args(where, delta, rg, q, k, v, g, beta, out, state_in, state_out,
                          state_index, device)
    _check(lib.dsa_gated_delta_decode(ctypes.byref(p), ctypes.byref(rg), *args,
                                      _raw_stream(stream, device)), where)


def dsa_device_status(clear: bool = True, stream=None) -> int:
    v = ctypes.c_int32(0)
    _check(lib.dsa_device_status(_stream(stream), ctypes.byref(v), int(clear)), "dsa_device_status")
    return v.value


def dsa_launch_count() -> int:
    return int(lib.dsa_launch_count())


def dsa_fused_rows(reset: bool = False) -> int:
    return int(lib.dsa_fused_rows(int(reset)))


def dsa_stage_timing(enable: bool):
    _check(lib.dsa_stage_timing(int(enable)), "dsa_stage_timing")


def dsa_stage_times(reset: bool = True):
    ms = (ctypes.c_double * 3)()
    n = (ctypes.c_int64 * 3)()
    _check(lib.dsa_stage_times(ms, n, int(reset)), "dsa_stage_times")
    return list(ms), list(n)


def workload_shape(w) -> LayerShape:
    """LayerShape of a dsa_synth.Workload."""
    return LayerShape(w.n_idx_heads, w.idx_dim, w.n_q_heads, w.n_kv_heads, w.head_dim, w.top_k,
                      DSA_FP8_E4M3 if w.idx_dtype == "fp8" else DSA_BF16)
