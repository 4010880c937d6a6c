"""Host-side checks of include/mqa_attend.h: the library exports it, the
binding's structure matches it, and bad arguments are refused before any
device memory is touched. No GPU needed (and nothing here launches work)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import fp8_mqa_logits_amd as mqa
from fp8_mqa_logits_amd import attend as A

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mqa_attend.h")

# fake, never-dereferenced device addresses (all checks fail before any use)
A16, MIS, WS = 0x10000, 0x10004, 0x20000
P = ctypes.c_void_p


def cache(**kw):
    a = dict(pages=A16, table=A16, page_stride=1 << 20, num_pages=4, table_stride=4, kv_heads=2,
             head_dim=128, page_size=64, block=64, codes=0)
    a.update(kw)
    return A._Cache(*(a[f] for f, _ in A._Cache._fields_))


def paged(c=None, **kw):
    a = dict(q=A16, q_row=1024, q_head=128, dtype=0, starts=A16, ends=A16, out=A16, lse=0,
             requests=1, R=4, heads=8, scale=1.0, ws=WS, wsb=1 << 40)
    a.update(kw)
    c = cache() if c is None else c
    return A._load().mqa_attend_paged(c, P(a["q"]), a["q_row"], a["q_head"], a["dtype"],
                                      P(a["starts"]), P(a["ends"]), P(a["out"]), P(a["lse"]),
                                      a["requests"], a["R"], a["heads"], a["scale"], P(a["ws"]),
                                      a["wsb"], None)


def topk(**kw):
    a = dict(idx=A16, width=512, q=A16, out=A16)
    a.update(kw)
    return A._load().mqa_attend_topk(cache(), P(a["q"]), 1024, 128, 0, P(a["idx"]), a["width"],
                                     P(A16), P(A16), P(a["out"]), None, 1, 4, 8, 1.0, P(WS),
                                     1 << 40, None)


def append(c=None, **kw):
    a = dict(k=A16, v=A16, kr=256, kh=128, vr=256, vh=128, dtype=0, starts=A16, counts=0,
             requests=1, R=4)
    a.update(kw)
    c = cache() if c is None else c
    return A._load().mqa_kv_append(c, P(a["k"]), a["kr"], a["kh"], P(a["v"]), a["vr"], a["vh"],
                                   a["dtype"], P(a["starts"]), P(a["counts"]), a["requests"],
                                   a["R"], None)


def test_exports_match_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^[a-z_][a-z0-9_ ]*[ *]+(\w+)\(", text, flags=re.M))
    assert names == set(mqa.ATTEND_EXPORTS)
    for n in names:
        assert hasattr(A._load(), n), n


def test_header_is_c_and_the_structure_is_the_bindings(tmp_path):
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "t.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "mqa_attend.h"\nint main(void) {'
                   + "".join(f'printf("%zu ", offsetof(mqa_kv_cache, {f}));' for f, _ in A._Cache._fields_)
                   + 'printf("%zu", sizeof(mqa_kv_cache)); return 0; }\n')
    exe = tmp_path / "t"
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                    str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    want = [getattr(A._Cache, f).offset for f, _ in A._Cache._fields_] + [ctypes.sizeof(A._Cache)]
    assert [int(x) for x in got] == want


def test_page_bytes():
    f = A._load().mqa_kv_page_bytes
    assert f(1, 64, 16, 16) == 2 * 16 * 64 + 128
    assert f(8, 128, 64, 64) == 2 * 8 * 64 * 128 + 128
    assert f(3, 128, 64, 16) == 2 * 3 * (64 * 128 + 16) + 32
    for bad in ((0, 128, 64, 64), (1025, 128, 64, 64), (1, 96, 64, 64), (1, 128, 48, 16),
                (1, 128, 8, 8), (1, 128, 64, 8), (1, 128, 64, 128), (1, 128, 64, 48),
                (1, 128, 1 << 17, 64), (1024, 128, 65536, 64)):
        assert f(*bad) == 0, bad


def test_attend_errors():
    for name in ("q", "starts", "ends", "out"):
        assert paged(**{name: 0}) == 1, name
    assert paged(cache(pages=0)) == 1
    assert paged(cache(table=0)) == 1
    for kw in (dict(q=0x10008), dict(out=MIS), dict(starts=0x10002), dict(lse=0x10002),
               dict(ws=0x20080), dict(q_row=1020), dict(q_head=132)):
        assert paged(**kw) == 2, kw
    assert paged(cache(pages=0x10008)) == 2
    assert paged(cache(page_stride=(1 << 20) + 8)) == 2
    for kw in (dict(requests=0), dict(R=0), dict(requests=1 << 11, R=1 << 10), dict(heads=7),
               dict(heads=0), dict(heads=1026), dict(dtype=2), dict(dtype=-1), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(q_row=-1024)):
        assert paged(**kw) == 3, kw
    for kw in (dict(page_stride=1024), dict(num_pages=0), dict(table_stride=0), dict(kv_heads=0),
               dict(head_dim=80), dict(page_size=24), dict(block=128), dict(codes=2)):
        assert paged(cache(**kw)) == 3, kw


def test_topk_errors():
    assert topk(idx=0) == 1
    assert topk(idx=0x10008) == 2
    assert topk(width=0) == 3
    assert topk(width=(1 << 16) + 1) == 3


def test_append_and_read_errors():
    for name in ("k", "v", "starts"):
        assert append(**{name: 0}) == 1, name
    for kw in (dict(k=0x10008), dict(v=0x10008), dict(starts=0x10002), dict(counts=0x10002),
               dict(kr=252), dict(vh=4)):
        assert append(**kw) == 2, kw
    for kw in (dict(requests=0), dict(R=0), dict(dtype=3), dict(kr=-256)):
        assert append(**kw) == 3, kw
    assert append(cache(kv_heads=0)) == 3
    L = A._load()
    assert L.mqa_kv_read(cache(), None, P(A16), 0, P(A16), None, 1, 4, None) == 1
    assert L.mqa_kv_read(cache(), P(A16), P(MIS), 0, P(A16), None, 1, 4, None) == 2
    assert L.mqa_kv_read(cache(), P(A16), P(A16), 3, P(A16), None, 1, 4, None) == 3
    assert L.mqa_kv_read(cache(), P(A16), P(A16), 0, P(A16), None, 1 << 20, 2, None) == 3


def test_no_device_is_an_error_not_a_fallback():
    import torch
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU")
    assert paged() == 5
    assert topk() == 5
    assert append() == 5
    assert A._load().workspace_size_attend(1, 1, 8, 2, 128, 512, 0) == 0
    with pytest.raises(ValueError):
        mqa.mqa_attend_paged(mqa.KVLayout(2, 128), torch.zeros(1, 8, 128, dtype=torch.bfloat16),
                             mqa.KVLayout(2, 128).alloc(2, "cpu"), torch.zeros(1, 1, dtype=torch.int32),
                             torch.zeros(1, dtype=torch.int32), torch.ones(1, dtype=torch.int32))


def test_a_layout_s_sizes_stay_those_of_its_page():
    # a cache is checked against the layout's page: sizes that change after that
    # would let a call past it into memory that is not the cache's
    L = mqa.KVLayout(2, 64, 16, 16)
    assert L.page_bytes == 2 * 2 * (16 * 64 + 4) + 112
    for field, value in (("kv_heads", 8), ("head_dim", 128), ("page_size", 64), ("block", 32),
                         ("codes", "int8")):
        with pytest.raises(AttributeError):
            setattr(L, field, value)
    assert mqa.KVLayout(2, 128, 16, 16).page_bytes == 2 * 2 * (16 * 128 + 4) + 112
    assert repr(L) == "KVLayout(kv_heads=2, head_dim=64, page_size=16, block=16, codes='e4m3')"
