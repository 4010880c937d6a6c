"""Python binding of what a serving step does around attention over the paged 8-bit
cache: norm and rotation of queries and keys, and eviction by accumulated attention
weight.

Argument marshalling only, as in the package's other entry points; the C ABI and its
contract are declared in include/mqa_serve.h. If the library is not built, every entry
point raises (there is no fallback).
"""
from __future__ import annotations

import ctypes
import math

import torch

from .attend import (DTYPES, NO_WORKSPACE, KVLayout, _Cache, _cache, _dense, _heads, _launch, _on,
                     _raise, _rows_per_request, _stream)

EXPORTS = ("mqa_norm_rotate", "mqa_kv_weigh", "workspace_size_weigh", "mqa_kv_select",
           "workspace_size_select",
           "mqa_kv_keep", "workspace_size_keep")


class _HeadRows(ctypes.Structure):
    """mqa_head_rows of include/mqa_serve.h."""
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


_bound = None


def _load() -> ctypes.CDLL:
    global _bound
    if _bound is None:
        from . import load
        lib = load()
        P, I, F, H = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.POINTER(_HeadRows)
        lib.mqa_norm_rotate.argtypes = [H, H, I, H, H, I, P, P, I, P, P, I, I, I, I, I, I, F, P]
        lib.mqa_norm_rotate.restype = I
        C, I64, SZ = ctypes.POINTER(_Cache), ctypes.c_int64, ctypes.c_size_t
        lib.mqa_kv_weigh.argtypes = [C, P, I64, I64, I, P, P, P, P, I, I, I, I, F, P, SZ, P]
        lib.mqa_kv_weigh.restype = I
        lib.workspace_size_weigh.argtypes = [I, I, I, I, I, I, I]
        lib.workspace_size_weigh.restype = SZ
        lib.mqa_kv_select.argtypes = [P, I, P, I, I, I, P, P, P, I, P, SZ, P]
        lib.mqa_kv_select.restype = I
        lib.workspace_size_select.argtypes = [I, I]
        lib.workspace_size_select.restype = SZ
        lib.mqa_kv_keep.argtypes = [C, P, P, P, I, I, P, SZ, P]
        lib.mqa_kv_keep.restype = I
        lib.workspace_size_keep.argtypes = [I, I, I, I, I]
        lib.workspace_size_keep.restype = SZ
        _bound = lib
    return _bound


def _head_rows(t, name, dtype, rows, heads, dim, dev):
    n, row, head = _heads(t, name, dtype, rows, heads, dim, dev)
    return n, _HeadRows(t.data_ptr(), row, head)


def mqa_norm_rotate(q, k, q_weight, k_weight, positions, inv_freq, eps: float | None = 1e-6,
                    pairs: bool = False, q_out=None, k_out=None, stream=None):
    """RMS norm of every query and key head (weights [head_dim] of q's dtype or fp32, None
    for ones; eps None: no norm), then the rotation by positions [rows] int32 times inv_freq
    [rot / 2] fp32 of its first rot elements, rot a multiple of 16 (None, both: no
    rotation): element i with i + rot / 2, or 2 i with 2 i + 1 where `pairs`. q [rows,
    heads, head_dim] and k [rows, kv_heads, head_dim] (None: no keys) in bf16 or fp16,
    head_dim 64, 128 or 256, any row and head strides. Returns (q_out, k_out): dense, unless
    given -- q and k themselves, or tensors that overlap nothing."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a tensor")
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"q: dtype {q.dtype}, expected bfloat16 or float16")
    if q.dim() != 3:
        raise ValueError(f"q: shape {tuple(q.shape)}, expected (rows, heads, head_dim)")
    dev, dtype, rows, dim = q.device, q.dtype, q.shape[0], q.shape[2]
    if dev.type != "cuda":
        raise ValueError("q must live on a GPU")
    heads, q_in = _head_rows(q, "q", dtype, rows, None, dim, dev)
    kv_heads, k_in = (0, None) if k is None else _head_rows(k, "k", dtype, rows, None, dim, dev)
    weight_type = dtype
    for t, name in ((q_weight, "q_weight"), (None if k is None else k_weight, "k_weight")):
        if t is not None:
            if isinstance(t, torch.Tensor) and t.dtype is torch.float32:
                weight_type = torch.float32
            _dense(t, name, weight_type, (dim,), dev)
    if q_weight is not None and q_weight.dtype is not weight_type:
        raise TypeError("q_weight and k_weight must be of one dtype")
    if eps is None and (q_weight is not None or k_weight is not None):
        raise ValueError("weights without a norm")
    rot = 0
    if (inv_freq is None) != (positions is None):
        raise TypeError("positions and inv_freq come together")
    if inv_freq is not None:
        _on(inv_freq, "inv_freq", torch.float32, dev)
        if inv_freq.dim() != 1 or not inv_freq.is_contiguous() or inv_freq.shape[0] == 0:
            raise ValueError("inv_freq must be contiguous, [rot / 2]")
        rot = 2 * inv_freq.shape[0]
        _dense(positions, "positions", torch.int32, (rows,), dev)
    with _launch(dev, stream):
        s = _stream(dev, stream)
        if q_out is None:
            q_out = torch.empty((rows, heads, dim), dtype=dtype, device=dev)
            q_to = _HeadRows(q_out.data_ptr(), heads * dim, dim)
        else:
            _, q_to = _head_rows(q_out, "q_out", dtype, rows, heads, dim, dev)
        if k is None:
            k_to = None
        elif k_out is None:
            k_out = torch.empty((rows, kv_heads, dim), dtype=dtype, device=dev)
            k_to = _HeadRows(k_out.data_ptr(), kv_heads * dim, dim)
        else:
            _, k_to = _head_rows(k_out, "k_out", dtype, rows, kv_heads, dim, dev)
        rc = _load().mqa_norm_rotate(
            q_in, q_to, heads, k_in, k_to, kv_heads, None if q_weight is None else q_weight.data_ptr(),
            None if k is None or k_weight is None else k_weight.data_ptr(), DTYPES[weight_type],
            None if rot == 0 else positions.data_ptr(), None if rot == 0 else inv_freq.data_ptr(), rot,
            int(pairs), rows, dim, DTYPES[dtype], int(eps is not None), 0.0 if eps is None else eps, s)
    _raise(rc, "mqa_norm_rotate")
    return q_out, (None if k is None else k_out)


def _workspace(t, dev):
    _on(t, "workspace", torch.uint8, dev)
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t


def workspace_size_weigh(requests: int, rows_per_request: int, heads: int, layout: KVLayout,
                         positions: int, device: int | None = None) -> int:
    """Bytes of workspace that suffice for every mqa_kv_weigh of up to so many requests, rows of
    each and positions (table_stride * page_size)."""
    if device is None:
        device = torch.cuda.current_device()
    return int(_load().workspace_size_weigh(int(requests), int(rows_per_request), int(heads),
                                            layout.kv_heads, layout.head_dim,
                                            min(int(positions), 1 << 20), int(device)))


def mqa_kv_weigh(layout: KVLayout, q, cache, page_table, starts, ends, lse, weights, scale=None,
                 workspace=None, stream=None) -> torch.Tensor:
    """Adds the attention weight that every position receives from a request's rows and
    heads, exp(score - lse), to weights [requests, width] fp32 (positions from width on are
    left out); returns weights. lse [requests * R, heads] fp32 as mqa_attend_paged returns it
    for the same q, starts, ends and scale (not that of a window or a tree, whose rows see
    other positions than their ranges); other arguments as there."""
    c, dev, requests = _cache(layout, cache, page_table)
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a tensor")
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"q: dtype {q.dtype}, expected bfloat16 or float16")
    rows = q.shape[0]
    heads, q_row, q_head = _heads(q, "q", q.dtype, rows, None, layout.head_dim, dev)
    R = _rows_per_request(rows, requests, "q")
    _dense(starts, "starts", torch.int32, (rows,), dev)
    _dense(ends, "ends", torch.int32, (rows,), dev)
    _dense(lse, "lse", torch.float32, (rows, heads), dev)
    if not isinstance(weights, torch.Tensor) or weights.dim() != 2:
        raise ValueError("weights must be a tensor [requests, width]")
    width = weights.shape[1]
    _dense(weights, "weights", torch.float32, (requests, width), dev)
    if scale is None:
        scale = 1.0 / math.sqrt(layout.head_dim)
    lib = _load()
    with _launch(dev, stream):
        s = _stream(dev, stream)
        if workspace is not None:
            _workspace(workspace, dev)
        else:
            n = lib.workspace_size_weigh(requests, R, heads, layout.kv_heads, layout.head_dim,
                                         min(c.table_stride * c.page_size, 1 << 20), dev.index)
            if n > NO_WORKSPACE:
                workspace = torch.empty(n, dtype=torch.uint8, device=dev)
        rc = lib.mqa_kv_weigh(c, q.data_ptr(), q_row, q_head, DTYPES[q.dtype], starts.data_ptr(),
                              ends.data_ptr(), lse.data_ptr(), weights.data_ptr(), width, requests, R,
                              heads, float(scale), None if workspace is None else workspace.data_ptr(),
                              0 if workspace is None else workspace.numel(), s)
    _raise(rc, "mqa_kv_weigh")
    return weights


def workspace_size_select(requests: int, width: int) -> int:
    """Bytes of workspace that suffice for every mqa_kv_select of up to so many requests and
    weights of each."""
    return int(_load().workspace_size_select(int(requests), int(width)))


def mqa_kv_select(weights, lengths, keep: int, sinks: int = 0, recent: int = 0, kept=None,
                  workspace=None, stream=None):
    """Which `keep` positions of each request stay: of its lengths[i] positions the first
    `sinks`, the last `recent` and the largest weights [requests, width] fp32 between them
    (equal ones: the smallest positions). Returns (positions [requests, keep] int32 in
    ascending order, -1 padded, counts [requests] int32). kept: a tensor like weights that
    takes the chosen positions' weights in that order, zeros behind them."""
    if not isinstance(weights, torch.Tensor) or weights.dim() != 2:
        raise ValueError("weights must be a tensor [requests, width]")
    dev, (requests, width) = weights.device, weights.shape
    if dev.type != "cuda":
        raise ValueError("weights must live on a GPU")
    _dense(weights, "weights", torch.float32, (requests, width), dev)
    _dense(lengths, "lengths", torch.int32, (requests,), dev)
    keep, sinks, recent = int(keep), int(sinks), int(recent)
    for name, n in (("keep", keep), ("sinks", sinks), ("recent", recent)):
        if not 0 <= n < 1 << 31:
            raise ValueError(f"{name}: {n} out of range")
    if kept is not None:
        _dense(kept, "kept", torch.float32, (requests, width), dev)
        if kept.data_ptr() == weights.data_ptr():
            raise ValueError("kept must be another tensor than weights")
    with _launch(dev, stream):
        s = _stream(dev, stream)
        positions = torch.empty((requests, keep), dtype=torch.int32, device=dev)
        counts = torch.empty(requests, dtype=torch.int32, device=dev)
        lib = _load()
        if workspace is not None:
            _workspace(workspace, dev)
        else:
            n = lib.workspace_size_select(requests, width)
            if n > NO_WORKSPACE:
                workspace = torch.empty(n, dtype=torch.uint8, device=dev)
        rc = lib.mqa_kv_select(weights.data_ptr(), width, lengths.data_ptr(), keep, sinks, recent,
                               positions.data_ptr(), counts.data_ptr(),
                               None if kept is None else kept.data_ptr(), requests,
                               None if workspace is None else workspace.data_ptr(),
                               0 if workspace is None else workspace.numel(), s)
    _raise(rc, "mqa_kv_select")
    return positions, counts


def workspace_size_keep(requests: int, width: int, layout: KVLayout) -> int:
    """Bytes of workspace that suffice for every mqa_kv_keep of up to so many requests and
    listed positions of each."""
    return int(_load().workspace_size_keep(int(requests), int(width), layout.kv_heads, layout.head_dim,
                                           layout.block))


def mqa_kv_keep(layout: KVLayout, cache, page_table, positions, counts, starts=None, workspace=None,
                stream=None) -> torch.Tensor:
    """Moves the first counts[i] listed positions [requests, width] int32 of every request
    (ascending; entry t none before starts[i] + t) to its positions starts[i] .. (int32; None:
    0 ..), as mqa_kv_append would store what mqa_kv_read returns for them in fp32: an eviction
    (mqa_kv_select's output), or the accepted tokens of a draft's tree. The request is
    starts[i] + counts[i] long afterwards. Writes and returns cache."""
    c, dev, requests = _cache(layout, cache, page_table)
    if not isinstance(positions, torch.Tensor) or positions.dim() != 2:
        raise ValueError("positions must be a tensor [requests, width]")
    width = positions.shape[1]
    _dense(positions, "positions", torch.int32, (requests, width), dev)
    _dense(counts, "counts", torch.int32, (requests,), dev)
    if starts is not None:
        _dense(starts, "starts", torch.int32, (requests,), dev)
    lib = _load()
    with _launch(dev, stream):
        s = _stream(dev, stream)
        if workspace is not None:
            _workspace(workspace, dev)
        else:
            n = lib.workspace_size_keep(requests, width, layout.kv_heads, layout.head_dim, layout.block)
            if n > NO_WORKSPACE:
                workspace = torch.empty(n, dtype=torch.uint8, device=dev)
        rc = lib.mqa_kv_keep(c, positions.data_ptr(), counts.data_ptr(),
                             None if starts is None else starts.data_ptr(), width, requests,
                             None if workspace is None else workspace.data_ptr(),
                             0 if workspace is None else workspace.numel(), s)
    _raise(rc, "mqa_kv_keep")
    return cache
