"""Python binding of the paged 8-bit key/value cache: storing tokens, reading
them back, and attention over ranges or listed positions of the cache.

Argument marshalling only, as in the package's other entry points; the C ABI
and its contract are declared in include/mqa_attend.h. If the library is not
built, every entry point raises (there is no fallback).
"""
from __future__ import annotations

import collections
import contextlib
import ctypes
import functools
import math

import torch

CODES = {"e4m3": 0, "int8": 1}
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
MAX_LIST = 1 << 16
NO_WORKSPACE = 256  # workspace_size_attend_call of a call that needs none

EXPORTS = ("mqa_kv_page_bytes", "mqa_kv_append", "mqa_kv_read", "workspace_size_attend",
           "workspace_size_attend_call", "mqa_attend_paged", "mqa_attend_topk")


class _Cache(ctypes.Structure):
    """mqa_kv_cache of include/mqa_attend.h."""
    _fields_ = [("pages", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("page_stride", ctypes.c_int64), ("num_pages", ctypes.c_int32),
                ("table_stride", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("block", ctypes.c_int32), ("codes", ctypes.c_int32)]


_bound = None


def _load() -> ctypes.CDLL:
    global _bound
    if _bound is None:
        from . import load
        lib = load()
        P, I, I64, SZ, F = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t,
                            ctypes.c_float)
        C = ctypes.POINTER(_Cache)
        lib.mqa_kv_page_bytes.argtypes = [I, I, I, I]
        lib.mqa_kv_page_bytes.restype = SZ
        lib.mqa_kv_append.argtypes = [C, P, I64, I64, P, I64, I64, I, P, P, I, I, P]
        lib.mqa_kv_append.restype = I
        lib.mqa_kv_read.argtypes = [C, P, P, I, P, P, I, I, P]
        lib.mqa_kv_read.restype = I
        lib.workspace_size_attend.argtypes = [I, I, I, I, I, I, I]
        lib.workspace_size_attend.restype = SZ
        lib.workspace_size_attend_call.argtypes = [I, I, I, I, I, I, I, I]
        lib.workspace_size_attend_call.restype = SZ
        lib.mqa_attend_paged.argtypes = [C, P, I64, I64, I, P, P, P, P, I, I, I, F, P, SZ, P]
        lib.mqa_attend_paged.restype = I
        lib.mqa_attend_topk.argtypes = [C, P, I64, I64, I, P, I, P, P, P, P, I, I, I, F, P, SZ, P]
        lib.mqa_attend_topk.restype = I
        _bound = lib
    return _bound


@functools.lru_cache(maxsize=None)
def _page_bytes(kv_heads: int, head_dim: int, page_size: int, block: int) -> int:
    return int(_load().mqa_kv_page_bytes(kv_heads, head_dim, page_size, block))


class KVLayout(collections.namedtuple("KVLayout", ("kv_heads", "head_dim", "page_size", "block",
                                                   "codes"))):
    """What a page of the cache holds: kv_heads key heads and as many value
    heads of head_dim (64 or 128) 8-bit codes ("e4m3" or "int8") for
    page_size tokens, and an fp32 scale for each block of tokens and head
    (page_size and block powers of two, 16 <= block <= page_size). Immutable."""
    __slots__ = ()

    def __new__(cls, kv_heads: int, head_dim: int, page_size: int = 64, block: int = 64,
                codes: str = "e4m3"):
        if codes not in CODES:
            raise ValueError(f"codes: {codes!r} not in {tuple(CODES)}")
        return super().__new__(cls, int(kv_heads), int(head_dim), int(page_size), int(block), codes)

    @property
    def page_bytes(self) -> int:
        """Bytes of a page; raises for sizes that no page can have."""
        n = _page_bytes(self.kv_heads, self.head_dim, self.page_size, self.block)
        if n == 0:
            raise ValueError(f"{self}: head_dim must be 64 or 128, page_size and block powers "
                             "of two, 16 <= block <= page_size <= 65536, a page below 2 GiB")
        return n

    def alloc(self, num_pages: int, device="cuda") -> torch.Tensor:
        """A zeroed pool of pages [num_pages, page_bytes] uint8."""
        return torch.zeros((num_pages, self.page_bytes), dtype=torch.uint8, device=device)


def _on(t, name: str, dtype, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} must live on {device}")


# (the checks below pass in one test; what fails it is told apart afterwards:
# a small call's time is the host's)

def _dense(t, name: str, dtype, shape: tuple, device):
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and \
            t.device == device and t.is_contiguous():
        return
    _on(t, name, dtype, device)
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
    raise ValueError(f"{name} must be contiguous")


def _heads(t, name: str, dtype, rows: int, heads: int | None, dim: int, device):
    """[rows, heads, dim] with a dense last axis; any row and head stride.
    Returns the shape's heads and the strides (0 for an axis of one element, whose
    stride torch leaves as it comes)."""
    _on(t, name, dtype, device)
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[0] != rows or shape[2] != dim or \
            (heads is not None and shape[1] != heads):
        raise ValueError(f"{name}: shape {tuple(shape)}, expected "
                         f"({rows}, {'heads' if heads is None else heads}, {dim})")
    if stride[2] != 1:
        raise ValueError(f"{name} must have a dense last axis")
    return shape[1], stride[0] if shape[0] > 1 else 0, stride[1] if shape[1] > 1 else 0


def _cache(layout: KVLayout, cache, page_table):
    if not isinstance(layout, KVLayout):
        raise TypeError("layout must be a KVLayout")
    if not isinstance(cache, torch.Tensor) or not isinstance(page_table, torch.Tensor):
        raise TypeError("cache and page_table must be tensors")
    dev = cache.device
    if dev.type != "cuda":
        raise ValueError("cache must live on a GPU")
    size, shape, stride = layout.page_bytes, cache.shape, cache.stride()
    if cache.dtype is not torch.uint8 or len(shape) != 2 or shape[1] != size or \
            stride[1] != 1 or (shape[0] > 1 and stride[0] < size):
        raise ValueError(f"cache must be [num_pages, {size}] uint8 with dense pages that do not "
                         "overlap")
    if page_table.dim() == 1:
        page_table = page_table[None]
    table = page_table.shape
    if len(table) != 2:
        raise ValueError("page_table must be [requests, table_stride] or [table_stride]")
    _dense(page_table, "page_table", torch.int32, table, dev)
    c = _Cache(cache.data_ptr(), page_table.data_ptr(), stride[0] if shape[0] > 1 else size,
               shape[0], table[1], layout.kv_heads, layout.head_dim, layout.page_size,
               layout.block, CODES[layout.codes])
    return c, dev, table[0]


def _rows_per_request(rows: int, requests: int, name: str) -> int:
    if requests < 1 or rows % requests:
        raise ValueError(f"{name} has {rows} rows, not a multiple of page_table's {requests} "
                         "requests")
    return rows // requests


def _raise(code: int, where: str):
    if code != 0:
        from . import MQAError
        raise MQAError(code, where)


@contextlib.contextmanager
def _elsewhere(dev, stream):
    with torch.cuda.device(dev):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


_HERE = contextlib.nullcontext()


def _launch(dev, stream):
    """The device made current and the stream that the call runs on; buffers
    that the binding allocates inside belong to that stream."""
    if stream is None and torch.cuda.current_device() == dev.index:
        return _HERE
    return _elsewhere(dev, stream)


def _stream(dev, stream) -> int:
    # torch.cuda.current_stream() builds a Stream object to the same end, at
    # a tenth of a small call's time
    return torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else stream.cuda_stream


def mqa_kv_append(layout: KVLayout, k, v, cache, page_table, starts, counts=None,
                  stream=None) -> torch.Tensor:
    """Store new tokens: k and v [requests * R, kv_heads, head_dim] (bf16, fp16
    or fp32; any row and head strides), row i * R + t being token t of request
    i, go to its positions starts[i] + t for t < counts[i] (int32; None: R).
    page_table [requests, table_stride] int32. The new tokens are the request's
    last: what their last block held behind them is lost. Writes and returns
    cache."""
    c, dev, requests = _cache(layout, cache, page_table)
    if not isinstance(k, torch.Tensor) or not isinstance(v, torch.Tensor):
        raise TypeError("k and v must be tensors")
    if k.dtype not in DTYPES:
        raise TypeError(f"k: dtype {k.dtype} not in {tuple(DTYPES)}")
    rows = k.shape[0]
    _, k_row, k_head = _heads(k, "k", k.dtype, rows, layout.kv_heads, layout.head_dim, dev)
    _, v_row, v_head = _heads(v, "v", k.dtype, rows, layout.kv_heads, layout.head_dim, dev)
    R = _rows_per_request(rows, requests, "k")
    _dense(starts, "starts", torch.int32, (requests,), dev)
    if counts is not None:
        _dense(counts, "counts", torch.int32, (requests,), dev)
    with _launch(dev, stream):
        s = _stream(dev, stream)
        rc = _load().mqa_kv_append(c, k.data_ptr(), k_row, k_head, v.data_ptr(), v_row, v_head,
                                   DTYPES[k.dtype], starts.data_ptr(),
                                   None if counts is None else counts.data_ptr(), requests, R, s)
    _raise(rc, "mqa_kv_append")
    return cache


def mqa_kv_read(layout: KVLayout, cache, page_table, starts, counts, rows_per_request: int,
                dtype=torch.bfloat16, out=None, stream=None):
    """Read positions starts[i] + t, t < counts[i] (int32; None: all R rows) of
    every request back as values: (k, v), each [requests * R, kv_heads,
    head_dim] of dtype, zero in the other rows. out: such a pair to write to."""
    c, dev, requests = _cache(layout, cache, page_table)
    R = int(rows_per_request)
    if R < 1:
        raise ValueError("rows_per_request must be at least 1")
    if dtype not in DTYPES:
        raise TypeError(f"dtype {dtype} not in {tuple(DTYPES)}")
    _dense(starts, "starts", torch.int32, (requests,), dev)
    if counts is not None:
        _dense(counts, "counts", torch.int32, (requests,), dev)
    shape = (requests * R, layout.kv_heads, layout.head_dim)
    with _launch(dev, stream):
        s = _stream(dev, stream)
        if out is None:
            out = (torch.empty(shape, dtype=dtype, device=dev),
                   torch.empty(shape, dtype=dtype, device=dev))
        else:
            _dense(out[0], "out[0]", dtype, shape, dev)
            _dense(out[1], "out[1]", dtype, shape, dev)
        rc = _load().mqa_kv_read(c, out[0].data_ptr(), out[1].data_ptr(), DTYPES[dtype],
                                 starts.data_ptr(), None if counts is None else counts.data_ptr(),
                                 requests, R, s)
    _raise(rc, "mqa_kv_read")
    return out[0], out[1]


def workspace_size_attend(requests: int, rows_per_request: int, heads: int, layout: KVLayout,
                          positions: int, device: int | None = None) -> int:
    """Bytes of workspace that suffice for every attention call of up to so many
    requests, rows of each and positions (table_stride * page_size for
    mqa_attend_paged, the list's width for mqa_attend_topk)."""
    if device is None:
        device = torch.cuda.current_device()
    return int(_load().workspace_size_attend(int(requests), int(rows_per_request), int(heads),
                                             layout.kv_heads, layout.head_dim,
                                             min(int(positions), 1 << 20), int(device)))


def _attend(layout, q, cache, page_table, indices, starts, ends, scale, out, lse, return_lse,
            workspace, stream, where):
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
    if indices is None:
        positions = min(c.table_stride * c.page_size, 1 << 20)
    else:
        if not isinstance(indices, torch.Tensor) or indices.dim() != 2:
            raise ValueError("indices must be a tensor [rows, width]")
        positions = indices.shape[1]
        _dense(indices, "indices", torch.int32, (rows, positions), dev)
    if scale is None:
        scale = 1.0 / math.sqrt(layout.head_dim)
    lib = _load()
    with _launch(dev, stream):
        s = _stream(dev, stream)
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        else:
            _dense(out, "out", q.dtype, (rows, heads, layout.head_dim), dev)
        if lse is not None:
            _dense(lse, "lse", torch.float32, (rows, heads), dev)
        elif return_lse:
            lse = torch.empty((rows, heads), dtype=torch.float32, device=dev)
        if workspace is None:
            n = lib.workspace_size_attend_call(requests, R, heads, layout.kv_heads,
                                               layout.head_dim, positions,
                                               int(indices is not None), dev.index)
            if n > NO_WORKSPACE:
                workspace = torch.empty(n, dtype=torch.uint8, device=dev)
        else:
            _on(workspace, "workspace", torch.uint8, dev)
            if not workspace.is_contiguous():
                raise ValueError("workspace must be contiguous")
        head = (c, q.data_ptr(), q_row, q_head, DTYPES[q.dtype])
        tail = (starts.data_ptr(), ends.data_ptr(), out.data_ptr(),
                None if lse is None else lse.data_ptr(), requests, R, heads, float(scale),
                None if workspace is None else workspace.data_ptr(),
                0 if workspace is None else workspace.numel(), s)
        if indices is None:
            rc = lib.mqa_attend_paged(*head, *tail)
        else:
            rc = lib.mqa_attend_topk(*head, indices.data_ptr(), positions, *tail)
    _raise(rc, where)
    return (out, lse) if return_lse else out


def mqa_attend_paged(layout: KVLayout, q, cache, page_table, starts, ends, scale=None, out=None,
                     lse=None, return_lse: bool = False, workspace=None, stream=None):
    """Attention of every row over positions [starts, ends) of its request:
    q [requests * R, heads, head_dim] bf16 or fp16 (any row and head strides;
    heads a multiple of layout.kv_heads), cache [num_pages, page_bytes] uint8
    (any page stride), page_table [requests, table_stride] int32 (or 1-D: one
    request), starts/ends [requests * R] int32. scale: of the scores, default
    1 / sqrt(head_dim). Returns out like q (dense), or (out, lse) with the rows'
    natural log-sum-exp [requests * R, heads] fp32. A row that sees nothing
    gives 0 and -inf."""
    return _attend(layout, q, cache, page_table, None, starts, ends, scale, out, lse, return_lse,
                   workspace, stream, "mqa_attend_paged")


def mqa_attend_topk(layout: KVLayout, q, cache, page_table, indices, starts, ends, scale=None,
                    out=None, lse=None, return_lse: bool = False, workspace=None, stream=None):
    """Attention of every row over its listed positions: indices [requests * R,
    width] int32 as mqa_topk_prefill_paged and mqa_topk_decode_paged return
    them (position - start, -1 padding) for the same starts and ends. Other
    arguments and results as mqa_attend_paged."""
    if indices is None:
        raise TypeError("indices must be a tensor")
    return _attend(layout, q, cache, page_table, indices, starts, ends, scale, out, lse,
                   return_lse, workspace, stream, "mqa_attend_topk")
