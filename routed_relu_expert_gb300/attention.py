"""Paged attention for verify blocks: the Python entry points of moe_paged_plan,
moe_rope, moe_rope_append and moe_tree_attention, of the calls for requests that
share pages (moe_paged_fork, moe_paged_compact, moe_paged_release,
moe_prefix_attention) and for rotary positions with several axes
(moe_rope_axes, moe_rope_append_axes), and a holder of one layer's paged KV cache.

As in ``layer``: each function checks tensor placement, types and shapes, takes
data pointers and the current CUDA stream, and calls the library, which launches
on the current device: the operands, and a stream that is given, have to be that
device's.  Rows ([T, heads, head_dim]) may be parts of a wider row, such as one
projection's q, k and v; caches are views [n_pages, page_size, n_kv_heads,
head_dim] of any layout whose head_dim is contiguous.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import struct
from dataclasses import dataclass
from typing import Optional, Sequence, Tuple

import torch

from . import _native as N
from .layer import _s

# the current stream's handle of a device, without building a Stream object for it (3 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)

_TORCH = {N.MOE_DT_BF16: torch.bfloat16, N.MOE_DT_F32: torch.float32}
# all fields of a moe_attn_config_t at once (reading them one by one costs as much as the launch)
_FIELDS = struct.Struct("@8ifi3q")
_SCALING = {None: N.MOE_ROPE_PLAIN, "linear": N.MOE_ROPE_LINEAR, "yarn": N.MOE_ROPE_YARN}


def make_attn_config(n_heads: int, n_kv_heads: int, head_dim: int, *, page_size: int = 16, n_pages: int = 0,
                     max_pages: int = 0, rot_dim: int = 0, rope_interleaved: bool = False,
                     softmax_scale: Optional[float] = None, dtype: int = N.MOE_DT_BF16,
                     k_cache: Optional[torch.Tensor] = None) -> N.MoeAttnConfig:
    """A moe_attn_config_t.  The cache's strides are those of ``k_cache``
    [n_pages, page_size, n_kv_heads, head_dim], or of a contiguous one;
    ``softmax_scale`` defaults to 1 / sqrt(head_dim)."""
    strides = ((page_size * n_kv_heads * head_dim, n_kv_heads * head_dim, head_dim) if k_cache is None
               else k_cache.stride()[:3])
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(head_dim) if head_dim > 0 else 1.0
    return N.MoeAttnConfig(n_heads, n_kv_heads, head_dim, page_size, n_pages, max_pages, rot_dim,
                           int(rope_interleaved), float(softmax_scale), dtype, *strides)


def _device(t: torch.Tensor, name: str) -> int:
    """The device that all of a call's tensors have to be on: that of ``t``, which is current."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev != _current_device():
        raise ValueError(f"{name} is on cuda:{dev}, the current device is cuda:{_current_device()}")
    return dev


def _stream(stream, dev: int):
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    if getattr(stream, "device_index", dev) != dev:
        raise ValueError(f"the stream is one of cuda:{stream.device_index}, the tensors are on cuda:{dev}")
    return _s(stream)


def attn_workspace_bytes(cfg: N.MoeAttnConfig) -> int:
    n = int(N.load().moe_attn_workspace_bytes(ctypes.byref(cfg)))
    if n == 0:
        N.check(N.load().moe_check_attn_config(ctypes.byref(cfg)), "moe_attn_workspace_bytes")
    return n


def new_attn_workspace(cfg: N.MoeAttnConfig, device="cuda") -> torch.Tensor:
    ws = torch.empty(attn_workspace_bytes(cfg), dtype=torch.uint8, device=device)
    ws[:N.MOE_ATTN_HEADER_BYTES].zero_()
    return ws


def prefix_workspace_bytes(cfg: N.MoeAttnConfig, T: int) -> int:
    n = int(N.load().moe_prefix_workspace_bytes(ctypes.byref(cfg), T))
    if n == 0:
        N.check(N.load().moe_check_attn_config(ctypes.byref(cfg)), "moe_prefix_workspace_bytes")
        raise ValueError(f"no workspace for {T} rows")
    return n


def new_prefix_workspace(cfg: N.MoeAttnConfig, T: int, device="cuda") -> torch.Tensor:
    """A workspace for moe_prefix_attention of up to T rows (it serves the other calls too)."""
    ws = torch.empty(prefix_workspace_bytes(cfg, T), dtype=torch.uint8, device=device)
    ws[:N.MOE_ATTN_HEADER_BYTES].zero_()
    return ws


def _array(t: Optional[torch.Tensor], dtype, n: Optional[int], name: str, dev: int):
    """Pointer of a contiguous array of n values (None: any number) on the device."""
    if t is None:
        return None
    if t.get_device() != dev or t.dtype is not dtype or not t.is_contiguous() or (n is not None and t.numel() != n):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on cuda:{dev}"
                         + ("" if n is None else f" of {n} values"))
    return t.data_ptr()


def _rows(t: torch.Tensor, T: int, heads: int, D: int, dt, name: str, dev: int) -> Tuple[int, int]:
    """(pointer, row stride) of rows [T, heads, D]."""
    if t.get_device() != dev or t.dtype is not dt or t.shape != (T, heads, D):
        raise ValueError(f"{name} must be a {dt} tensor on cuda:{dev} of shape {(T, heads, D)}")
    ld, step, one = t.stride()
    if (one != 1 and D > 1) or (heads > 1 and step != D):
        raise ValueError(f"the heads of a row of {name} must be contiguous")
    return t.data_ptr(), (ld if T > 1 else heads * D)


def _cache(t: torch.Tensor, shape, strides, dt, name: str, dev: int) -> int:
    if t.get_device() != dev or t.dtype is not dt or t.shape != shape:
        raise ValueError(f"{name} must be a {dt} tensor on cuda:{dev} of shape {shape}")
    if t.stride() != strides:
        raise ValueError(f"{name} does not have the configuration's strides")
    return t.data_ptr()


def _words(tree_mask: Optional[torch.Tensor], T: int) -> int:
    """Words a row of the mask (0: no mask, chains)."""
    if tree_mask is None:
        return 0
    shape = tree_mask.shape
    if len(shape) != 2 or shape[0] != T or shape[1] < 1:
        raise ValueError(f"tree_mask must be of shape ({T}, words)")
    return shape[1]


def moe_paged_plan(cfg, ctx_len, new_len, block_table, free_pages, free_head, q_start, kv_len, positions, slot_map,
                   ws, free_head_out=None, parents=None, tree_mask=None, stream=None):
    """Block tables, slots, positions and tree masks of a step, written into
    block_table, q_start, kv_len, positions, slot_map, tree_mask and
    free_head_out (default: free_head, in place)."""
    dev, R, T, i32 = _device(ws, "ws"), ctx_len.shape[0], positions.shape[0], torch.int32
    words = _words(tree_mask, T)
    N.check(N.load().moe_paged_plan(
        ctypes.byref(cfg), R, T, _array(ctx_len, i32, R, "ctx_len", dev), _array(new_len, i32, R, "new_len", dev),
        _array(parents, i32, T, "parents", dev), _array(block_table, i32, R * cfg.max_pages, "block_table", dev),
        _array(free_pages, i32, None, "free_pages", dev), free_pages.numel(),
        _array(free_head, i32, 1, "free_head", dev),
        _array(free_head if free_head_out is None else free_head_out, i32, 1, "free_head_out", dev),
        _array(q_start, i32, R + 1, "q_start", dev), _array(kv_len, i32, R, "kv_len", dev),
        _array(positions, i32, T, "positions", dev), _array(slot_map, torch.int64, T, "slot_map", dev),
        _array(tree_mask, i32, T * words, "tree_mask", dev), words,
        _array(ws, torch.uint8, None, "ws", dev), ws.numel(), _stream(stream, dev)), "moe_paged_plan")


def rope_table(rot_dim: int, theta: float, *, scaling: Optional[str] = None, factor: float = 1.0,
               original_context: int = 0, device="cuda") -> Tuple[torch.Tensor, float]:
    """(table on ``device``, rot_scale) of moe_rope_table; scaling: None, "linear" or "yarn"."""
    if scaling not in _SCALING:
        raise ValueError(f"unknown rotary scaling {scaling!r}")
    host = torch.zeros(max(rot_dim // 2, 1), dtype=torch.int64)
    scale = ctypes.c_float(1.0)
    N.check(N.load().moe_rope_table(rot_dim, float(theta), _SCALING[scaling], float(factor), int(original_context),
                                    host.data_ptr(), ctypes.byref(scale)), "moe_rope_table")
    return host.to(device), float(scale.value)


def _table(rot: int, table, dev: int):
    if rot == 0:
        return None
    if table is None:
        raise ValueError("table is missing")
    return _array(table, torch.int64, rot // 2, "table", dev)


def moe_rope(cfg, x, positions, table, out, rot_scale: float = 1.0, inverse: bool = False, stream=None):
    """Rows x [T, heads, head_dim] turned by their positions into ``out`` (which
    may be x); ``inverse`` is the backward."""
    dev, T, heads = _device(x, "x"), x.shape[0], x.shape[1]
    _, _, D, _, _, _, rot, _, _, dtype, _, _, _ = _FIELDS.unpack_from(cfg)
    dt = _TORCH.get(dtype)
    xp, x_ld = _rows(x, T, heads, D, dt, "x", dev)
    op, o_ld = _rows(out, T, heads, D, dt, "out", dev)
    N.check(N.load().moe_rope(ctypes.byref(cfg), T, heads, xp, x_ld,
                              _array(positions, torch.int32, T, "positions", dev), _table(rot, table, dev), rot_scale,
                              int(inverse), op, o_ld, _stream(stream, dev)), "moe_rope")


def moe_rope_append(cfg, q, k, v, positions, table, slot_map, k_cache, v_cache, q_out, ws, rot_scale: float = 1.0,
                    stream=None):
    """q turned into q_out (which may be q); k turned and v as it is into the
    caches at slot_map."""
    dev, T = _device(ws, "ws"), q.shape[0]
    H, Hkv, D, page, pages, _, rot, _, _, dtype, sp, st, sh = _FIELDS.unpack_from(cfg)
    dt = _TORCH.get(dtype)
    qp, q_ld = _rows(q, T, H, D, dt, "q", dev)
    kp, k_ld = _rows(k, T, Hkv, D, dt, "k", dev)
    vp, v_ld = _rows(v, T, Hkv, D, dt, "v", dev)
    op, o_ld = _rows(q_out, T, H, D, dt, "q_out", dev)
    shape, strides = (pages, page, Hkv, D), (sp, st, sh, 1)
    N.check(N.load().moe_rope_append(ctypes.byref(cfg), T, qp, q_ld, kp, k_ld, vp, v_ld,
                                     _array(positions, torch.int32, T, "positions", dev), _table(rot, table, dev),
                                     rot_scale, _array(slot_map, torch.int64, T, "slot_map", dev), op, o_ld,
                                     _cache(k_cache, shape, strides, dt, "k_cache", dev),
                                     _cache(v_cache, shape, strides, dt, "v_cache", dev),
                                     _array(ws, torch.uint8, None, "ws", dev), ws.numel(), _stream(stream, dev)),
            "moe_rope_append")


def rope_axes_table(sections: Sequence[int], theta: float, *, interleaved: bool = False, own_ladders: bool = False,
                    scaling: Optional[str] = None, factor: float = 1.0, original_context: int = 0,
                    device="cuda") -> Tuple[torch.Tensor, torch.Tensor, float]:
    """(table, axis of each pair, both on ``device``; rot_scale) of
    moe_rope_axes_table: sections[a] pairs turn by axis a."""
    if scaling not in _SCALING:
        raise ValueError(f"unknown rotary scaling {scaling!r}")
    n = (ctypes.c_int32 * max(len(sections), 1))(*sections)
    half = max(sum(sections), 1)
    if not 1 <= half <= 64:
        raise ValueError(f"sections {tuple(sections)} must have at most 64 pairs in all")
    table, axis = torch.zeros(half, dtype=torch.int64), torch.zeros(half, dtype=torch.uint8)
    scale = ctypes.c_float(1.0)
    N.check(N.load().moe_rope_axes_table(len(sections), n, int(interleaved), int(own_ladders), float(theta),
                                         _SCALING[scaling], float(factor), int(original_context), table.data_ptr(),
                                         axis.data_ptr(), ctypes.byref(scale)), "moe_rope_axes_table")
    return table.to(device), axis.to(device), float(scale.value)


def _axes(rot: int, positions, axis, T: int, dev: int):
    """(number of axes, pointers of positions [axes, T] and of the pairs' axes)."""
    if len(positions.shape) != 2:
        raise ValueError(f"positions must be of shape (axes, {T})")
    n = positions.shape[0]
    if rot and axis is None:
        raise ValueError("axis is missing")
    return (n, _array(positions, torch.int32, n * T, "positions", dev),
            _array(axis, torch.uint8, rot // 2, "axis", dev) if rot else None)


def moe_rope_axes(cfg, x, positions, axis, table, out, rot_scale: float = 1.0, inverse: bool = False, stream=None):
    """moe_rope with positions [axes, T]; ``axis`` and ``table`` are rope_axes_table's."""
    dev, T, heads = _device(x, "x"), x.shape[0], x.shape[1]
    _, _, D, _, _, _, rot, _, _, dtype, _, _, _ = _FIELDS.unpack_from(cfg)
    dt = _TORCH.get(dtype)
    xp, x_ld = _rows(x, T, heads, D, dt, "x", dev)
    op, o_ld = _rows(out, T, heads, D, dt, "out", dev)
    N.check(N.load().moe_rope_axes(ctypes.byref(cfg), T, heads, xp, x_ld, *_axes(rot, positions, axis, T, dev),
                                   _table(rot, table, dev), rot_scale, int(inverse), op, o_ld, _stream(stream, dev)),
            "moe_rope_axes")


def moe_rope_append_axes(cfg, q, k, v, positions, axis, table, slot_map, k_cache, v_cache, q_out, ws,
                         rot_scale: float = 1.0, stream=None):
    """moe_rope_append with positions [axes, T]; ``axis`` and ``table`` are rope_axes_table's."""
    dev, T = _device(ws, "ws"), q.shape[0]
    H, Hkv, D, page, pages, _, rot, _, _, dtype, sp, st, sh = _FIELDS.unpack_from(cfg)
    dt = _TORCH.get(dtype)
    qp, q_ld = _rows(q, T, H, D, dt, "q", dev)
    kp, k_ld = _rows(k, T, Hkv, D, dt, "k", dev)
    vp, v_ld = _rows(v, T, Hkv, D, dt, "v", dev)
    op, o_ld = _rows(q_out, T, H, D, dt, "q_out", dev)
    shape, strides = (pages, page, Hkv, D), (sp, st, sh, 1)
    N.check(N.load().moe_rope_append_axes(ctypes.byref(cfg), T, qp, q_ld, kp, k_ld, vp, v_ld,
                                          *_axes(rot, positions, axis, T, dev), _table(rot, table, dev), rot_scale,
                                          _array(slot_map, torch.int64, T, "slot_map", dev), op, o_ld,
                                          _cache(k_cache, shape, strides, dt, "k_cache", dev),
                                          _cache(v_cache, shape, strides, dt, "v_cache", dev),
                                          _array(ws, torch.uint8, None, "ws", dev), ws.numel(), _stream(stream, dev)),
            "moe_rope_append_axes")


def moe_tree_attention(cfg, q, q_start, kv_len, block_table, k_cache, v_cache, out, ws, tree_mask=None, lse=None,
                       stream=None):
    """out [T, n_heads, head_dim] (and lse [T, n_heads] FP32) of the rows q over the cache."""
    dev, T, R, i32 = _device(ws, "ws"), q.shape[0], kv_len.shape[0], torch.int32
    H, Hkv, D, page, pages, max_pages, _, _, _, dtype, sp, st, sh = _FIELDS.unpack_from(cfg)
    dt = _TORCH.get(dtype)
    words = _words(tree_mask, T)
    qp, q_ld = _rows(q, T, H, D, dt, "q", dev)
    op, o_ld = _rows(out, T, H, D, dt, "out", dev)
    shape, strides = (pages, page, Hkv, D), (sp, st, sh, 1)
    N.check(N.load().moe_tree_attention(
        ctypes.byref(cfg), R, T, qp, q_ld, _array(q_start, i32, R + 1, "q_start", dev),
        _array(kv_len, i32, R, "kv_len", dev), _array(block_table, i32, R * max_pages, "block_table", dev),
        _cache(k_cache, shape, strides, dt, "k_cache", dev), _cache(v_cache, shape, strides, dt, "v_cache", dev),
        _array(tree_mask, i32, T * words, "tree_mask", dev), words, op, o_ld,
        _array(lse, torch.float32, T * H, "lse", dev), _array(ws, torch.uint8, None, "ws", dev), ws.numel(),
        _stream(stream, dev)), "moe_tree_attention")


def moe_prefix_attention(cfg, q, q_start, kv_len, block_table, group_start, prefix_row, prefix_len, k_cache, v_cache,
                         out, ws, tree_mask=None, lse=None, stream=None):
    """moe_tree_attention where group g, requests group_start[g] .. group_start[g + 1] - 1,
    has its first prefix_len[g] tokens in common, in the pages of row prefix_row[g] of the
    table: they are attended once for the group's rows."""
    dev, T, R, i32 = _device(ws, "ws"), q.shape[0], kv_len.shape[0], torch.int32
    H, Hkv, D, page, pages, max_pages, _, _, _, dtype, sp, st, sh = _FIELDS.unpack_from(cfg)
    dt = _TORCH.get(dtype)
    words, groups = _words(tree_mask, T), prefix_len.numel()
    qp, q_ld = _rows(q, T, H, D, dt, "q", dev)
    op, o_ld = _rows(out, T, H, D, dt, "out", dev)
    shape, strides = (pages, page, Hkv, D), (sp, st, sh, 1)
    N.check(N.load().moe_prefix_attention(
        ctypes.byref(cfg), R, T, qp, q_ld, _array(q_start, i32, R + 1, "q_start", dev),
        _array(kv_len, i32, R, "kv_len", dev), _array(block_table, i32, R * max_pages, "block_table", dev), groups,
        _array(group_start, i32, groups + 1, "group_start", dev), _array(prefix_row, i32, groups, "prefix_row", dev),
        _array(prefix_len, i32, groups, "prefix_len", dev), _cache(k_cache, shape, strides, dt, "k_cache", dev),
        _cache(v_cache, shape, strides, dt, "v_cache", dev), _array(tree_mask, i32, T * words, "tree_mask", dev), words,
        op, o_ld, _array(lse, torch.float32, T * H, "lse", dev), _array(ws, torch.uint8, None, "ws", dev), ws.numel(),
        _stream(stream, dev)), "moe_prefix_attention")


def moe_paged_fork(cfg, src_rows, dst_rows, lengths, block_table, page_shares, free_pages, free_head, k_cache, v_cache,
                   ws, free_head_out=None, dst_table=None, stream=None):
    """Row dst_rows[i] of dst_table (default: block_table, the sources') goes on from the
    first lengths[i] tokens of row src_rows[i]: whole pages shared, the last one's tokens
    copied.  Written: dst_table, page_shares, the caches, free_head_out (default:
    free_head, in place).  One layer's K and V: of layers that share a table the others follow
    with the same free_head, their caches, and a dst_table, page_shares and free_head_out that
    nobody reads."""
    dev, n, R, i32 = _device(ws, "ws"), src_rows.shape[0], block_table.shape[0], torch.int32
    _, Hkv, D, page, pages, max_pages, _, _, _, dtype, sp, st, sh = _FIELDS.unpack_from(cfg)
    dt = _TORCH.get(dtype)
    shape, strides = (pages, page, Hkv, D), (sp, st, sh, 1)
    N.check(N.load().moe_paged_fork(
        ctypes.byref(cfg), n, _array(src_rows, i32, n, "src_rows", dev), _array(dst_rows, i32, n, "dst_rows", dev),
        _array(lengths, i32, n, "lengths", dev), R, _array(block_table, i32, R * max_pages, "block_table", dev),
        _array(block_table if dst_table is None else dst_table, i32, R * max_pages, "dst_table", dev),
        _array(page_shares, i32, pages, "page_shares", dev), _array(free_pages, i32, None, "free_pages", dev),
        free_pages.numel(), _array(free_head, i32, 1, "free_head", dev),
        _array(free_head if free_head_out is None else free_head_out, i32, 1, "free_head_out", dev),
        _cache(k_cache, shape, strides, dt, "k_cache", dev), _cache(v_cache, shape, strides, dt, "v_cache", dev),
        _array(ws, torch.uint8, None, "ws", dev), ws.numel(), _stream(stream, dev)), "moe_paged_fork")


def moe_paged_compact(cfg, first, keep_start, keep, block_table, k_cache, v_cache, ws, page_shares=None, len_out=None,
                      stream=None):
    """Of request r's tokens from first[r] on, numbers keep[keep_start[r]:keep_start[r + 1]]
    (ascending) move to the front, K and V, in place; len_out [R]: the tokens then."""
    dev, R, i32 = _device(ws, "ws"), first.shape[0], torch.int32
    _, Hkv, D, page, pages, max_pages, _, _, _, dtype, sp, st, sh = _FIELDS.unpack_from(cfg)
    dt = _TORCH.get(dtype)
    shape, strides = (pages, page, Hkv, D), (sp, st, sh, 1)
    N.check(N.load().moe_paged_compact(
        ctypes.byref(cfg), R, keep.numel(), _array(first, i32, R, "first", dev),
        _array(keep_start, i32, R + 1, "keep_start", dev), _array(keep, i32, None, "keep", dev),
        _array(block_table, i32, R * max_pages, "block_table", dev),
        _array(page_shares, i32, pages, "page_shares", dev), _array(len_out, i32, R, "len_out", dev),
        _cache(k_cache, shape, strides, dt, "k_cache", dev), _cache(v_cache, shape, strides, dt, "v_cache", dev),
        _array(ws, torch.uint8, None, "ws", dev), ws.numel(), _stream(stream, dev)), "moe_paged_compact")


def moe_paged_release(cfg, held_len, keep_len, block_table, free_pages, free_head, ws, page_shares=None, stream=None):
    """Gives back the pages of request r's first held_len[r] tokens that its first
    keep_len[r] do not need; block_table, page_shares, free_pages and free_head change in place."""
    dev, R, i32 = _device(ws, "ws"), held_len.shape[0], torch.int32
    _, _, _, _, pages, max_pages, _, _, _, _, _, _, _ = _FIELDS.unpack_from(cfg)
    N.check(N.load().moe_paged_release(
        ctypes.byref(cfg), R, _array(held_len, i32, R, "held_len", dev), _array(keep_len, i32, R, "keep_len", dev),
        _array(block_table, i32, R * max_pages, "block_table", dev),
        _array(page_shares, i32, pages, "page_shares", dev), _array(free_pages, i32, None, "free_pages", dev),
        free_pages.numel(), _array(free_head, i32, 1, "free_head", dev), _array(ws, torch.uint8, None, "ws", dev),
        ws.numel(), _stream(stream, dev)), "moe_paged_release")


def _memory_of(stream, device):
    """Within it, new tensors are the memory of the stream that a call is given (None: the current one)."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device) if int(stream) else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


@dataclass
class PagedStep:
    """What PagedKVCache.plan leaves for the other calls of a step."""
    q_start: torch.Tensor               # [R + 1]
    kv_len: torch.Tensor                # [R]
    positions: torch.Tensor             # [T]
    slot_map: torch.Tensor              # [T]
    tree_mask: Optional[torch.Tensor]   # [T, words]


@dataclass
class PrefixGroups:
    """Requests with common prefixes, for PagedKVCache.attend: group g is requests
    start[g] .. start[g + 1] - 1, which have their first length[g] tokens in common, in the
    pages of row row[g] of the block table (one of theirs, or a row that only holds the
    prefix).  int32, on the device."""
    start: torch.Tensor                 # [groups + 1]
    row: torch.Tensor                   # [groups]
    length: torch.Tensor                # [groups]


class PagedKVCache:
    """One attention layer's paged KV cache: the pages, the requests' block
    tables, the free pages, the holders of shared pages and the workspace (``ws``, with the
    error word that moe_get_device_error reads).  A step is plan -> append -> attend, all on the
    current stream, nothing on the host.  A call that is given another
    stream makes its tensors from that stream's memory; they are used on a third one
    as any tensor is (after an event, with ``record_stream``).  All calls share ``ws``:
    those on different streams are ordered by the caller, but ``release`` may run beside
    the ``append`` and ``attend`` of requests that keep what they have.

    ``prefix_rows``: rows of the largest step that ``attend`` gets groups for, of 2048 requests at
    most (it sizes the workspace: some 95 MB and the rows' own for BF16 heads of 128, 21 MB
    without it).  Caches of one configuration whose calls are ordered may have one workspace: set
    ``ws`` of the others to the first one's.  ``sections``: pairs a rotary axis, for positions with several
    (``interleaved_axes``, ``own_ladders``: as in rope_axes_table)."""

    def __init__(self, cfg: N.MoeAttnConfig, max_requests: int, device="cuda", theta: float = 10000.0, *,
                 prefix_rows: int = 0, sections: Optional[Sequence[int]] = None, interleaved_axes: bool = False,
                 own_ladders: bool = False, **scaling):
        if sections is not None and 2 * sum(sections) != cfg.rot_dim:
            raise ValueError(f"sections {tuple(sections)} must have rot_dim / 2 = {cfg.rot_dim // 2} pairs")
        self.cfg = cfg
        shape = (cfg.n_pages, cfg.page_size, cfg.n_kv_heads, cfg.head_dim)
        dt = _TORCH[cfg.dtype]
        self.k_cache = torch.zeros(shape, dtype=dt, device=device)
        self.v_cache = torch.zeros(shape, dtype=dt, device=device)
        self.block_table = torch.full((max_requests, cfg.max_pages), -1, dtype=torch.int32, device=device)
        self.free_pages = torch.arange(cfg.n_pages, dtype=torch.int32, device=device)
        self.free_head = torch.zeros(1, dtype=torch.int32, device=device)
        self.page_shares = torch.zeros(cfg.n_pages, dtype=torch.int32, device=device)
        self.ws = new_prefix_workspace(cfg, prefix_rows, device) if prefix_rows else new_attn_workspace(cfg, device)
        self.axes, self.axis = 1, None
        if sections is None:
            self.table, self.rot_scale = rope_table(cfg.rot_dim, theta, device=device, **scaling)
        else:
            self.axes = len(sections)
            self.table, self.axis, self.rot_scale = rope_axes_table(
                sections, theta, interleaved=interleaved_axes, own_ladders=own_ladders, device=device, **scaling)

    def plan(self, ctx_len, new_len, T: int, parents=None, max_nodes: Optional[int] = None, stream=None) -> PagedStep:
        """ctx_len, new_len [R] (R = max_requests; idle requests bring 0 tokens);
        T rows; parents [T]: trees of up to max_nodes nodes (nodes past that are seen by
        nobody, with MOE_DEVERR_CACHE in the workspace's error word).  By default the mask
        has room for any tree that T rows and a block-table row can hold; a server with
        many rows passes its largest tree, for T * ceil(max_nodes / 32) words of mask."""
        R, dev = self.block_table.shape[0], self.block_table.device
        if max_nodes is None:
            max_nodes = max(1, min(T, self.cfg.max_pages * self.cfg.page_size))
        elif max_nodes < 1:
            raise ValueError(f"max_nodes must be at least 1, got {max_nodes}")

        def new(*shape, dtype=torch.int32):
            return torch.empty(shape, dtype=dtype, device=dev)

        with _memory_of(stream, dev):
            step = PagedStep(new(R + 1), new(R), new(T), new(T, dtype=torch.int64),
                             None if parents is None else new(T, -(-max_nodes // 32)))
        moe_paged_plan(self.cfg, ctx_len, new_len, self.block_table, self.free_pages, self.free_head, step.q_start,
                       step.kv_len, step.positions, step.slot_map, self.ws, parents=parents,
                       tree_mask=step.tree_mask, stream=stream)
        return step

    def append(self, step: PagedStep, q, k, v, q_out=None, stream=None, positions=None) -> torch.Tensor:
        """Rotated queries; the keys and values of the step are in the cache after it.
        ``positions`` [axes, T] int32 for a cache with several axes (default: the step's own,
        as text has them, on every axis), [T] for one with one."""
        with _memory_of(stream, q.device):
            if q_out is None:
                q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            if positions is None:
                positions = step.positions if self.axis is None else step.positions.repeat(self.axes, 1)
        if self.axis is not None:
            if positions.shape[0] != self.axes:
                raise ValueError(f"positions must be of shape ({self.axes}, {q.shape[0]})")
            moe_rope_append_axes(self.cfg, q, k, v, positions, self.axis, self.table, step.slot_map, self.k_cache,
                                 self.v_cache, q_out, self.ws, rot_scale=self.rot_scale, stream=stream)
            return q_out
        moe_rope_append(self.cfg, q, k, v, positions, self.table, step.slot_map, self.k_cache, self.v_cache,
                        q_out, self.ws, rot_scale=self.rot_scale, stream=stream)
        return q_out

    def attend(self, step: PagedStep, q, out=None, lse=None, stream=None,
               groups: Optional[PrefixGroups] = None) -> torch.Tensor:
        """``groups``: the requests' common prefixes, attended once for each group."""
        if out is None:
            with _memory_of(stream, q.device):
                out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if groups is not None:
            moe_prefix_attention(self.cfg, q, step.q_start, step.kv_len, self.block_table, groups.start, groups.row,
                                 groups.length, self.k_cache, self.v_cache, out, self.ws, tree_mask=step.tree_mask,
                                 lse=lse, stream=stream)
            return out
        moe_tree_attention(self.cfg, q, step.q_start, step.kv_len, self.block_table, self.k_cache, self.v_cache, out,
                           self.ws, tree_mask=step.tree_mask, lse=lse, stream=stream)
        return out

    def fork(self, src_rows, dst_rows, lengths, stream=None) -> None:
        """Rows dst_rows of the block table (int32, holding nothing) go on from the first
        ``lengths`` tokens of rows src_rows: whole pages are shared, a partly filled last one
        is copied."""
        moe_paged_fork(self.cfg, src_rows, dst_rows, lengths, self.block_table, self.page_shares, self.free_pages,
                       self.free_head, self.k_cache, self.v_cache, self.ws, stream=stream)

    def compact(self, first, keep_start, keep, len_out=None, stream=None) -> torch.Tensor:
        """Moves the kept tokens of each request (numbers from ``first`` on, ascending: the
        nodes of an accepted path, say) to the front; the requests' lengths then."""
        if len_out is None:
            with _memory_of(stream, first.device):
                len_out = torch.empty(first.shape[0], dtype=torch.int32, device=first.device)
        moe_paged_compact(self.cfg, first, keep_start, keep, self.block_table, self.k_cache, self.v_cache, self.ws,
                          page_shares=self.page_shares, len_out=len_out, stream=stream)
        return len_out

    def release(self, kv_len: torch.Tensor, ctx_len: torch.Tensor, stream=None) -> None:
        """Gives the pages back that a request holds for its first kv_len tokens but not
        for its first ctx_len (a rejected part of a draft; 0: a finished request).  They
        go before the list's head, which the next plan takes pages from; a page that others
        hold too only loses a holder.  kv_len, ctx_len [R]; nothing on the host."""
        dev = self.block_table.device
        with torch.cuda.device(dev), _memory_of(stream, dev):
            kv_len, ctx_len = (n.to(torch.int32).contiguous() for n in (kv_len, ctx_len))
            moe_paged_release(self.cfg, kv_len, ctx_len, self.block_table, self.free_pages, self.free_head, self.ws,
                              page_shares=self.page_shares, stream=stream)
