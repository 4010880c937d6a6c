"""Python binding of what a serving step does around attention over the paged 8-bit
cache: norm and rotation of queries and keys.

Argument marshalling only, as in the package's other entry points; the C ABI and its
contract are declared in include/mqa_serve.h. If the library is not built, every entry
point raises (there is no fallback).
"""
from __future__ import annotations

import ctypes

import torch

from .attend import DTYPES, _dense, _heads, _launch, _on, _raise, _stream

EXPORTS = ("mqa_norm_rotate",)


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
            q_out = torch.empty(q.shape, dtype=dtype, device=dev)
        if k_out is None and k is not None:
            k_out = torch.empty(k.shape, dtype=dtype, device=dev)
        _, q_to = _head_rows(q_out, "q_out", dtype, rows, heads, dim, dev)
        k_to = None if k is None else _head_rows(k_out, "k_out", dtype, rows, kv_heads, dim, dev)[1]
        rc = _load().mqa_norm_rotate(
            q_in, q_to, heads, k_in, k_to, kv_heads, None if q_weight is None else q_weight.data_ptr(),
            None if k is None or k_weight is None else k_weight.data_ptr(), DTYPES[weight_type],
            None if rot == 0 else positions.data_ptr(), None if rot == 0 else inv_freq.data_ptr(), rot,
            int(pairs), rows, dim, DTYPES[dtype], int(eps is not None), 0.0 if eps is None else eps, s)
    _raise(rc, "mqa_norm_rotate")
    return q_out, (None if k is None else k_out)
