"""Host-side checks of what a serving step does around attention: bad arguments are
refused before any device memory is touched. No GPU needed (nothing here launches
work; the addresses are never used)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import fp8_mqa_logits_amd as mqa
from fp8_mqa_logits_amd import attend as A
from fp8_mqa_logits_amd import serve as S
from test_attend_host import A16, MIS, WS, cache

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p


def window(c=None, **kw):
    a = dict(q=A16, q_row=1024, q_head=128, dtype=0, starts=A16, ends=A16, window=100, sinks=4,
             out=A16, lse=0, requests=1, R=4, heads=8, scale=1.0, ws=WS, wsb=1 << 40)
    assert set(kw) <= set(a)
    a.update(kw)
    return A._load().mqa_attend_window(
        cache() if c is None else c, P(a["q"]), a["q_row"], a["q_head"], a["dtype"], P(a["starts"]),
        P(a["ends"]), a["window"], a["sinks"], P(a["out"]), P(a["lse"]), a["requests"], a["R"],
        a["heads"], a["scale"], P(a["ws"]), a["wsb"], None)


def tree(c=None, **kw):
    a = dict(q=A16, q_row=1024, q_head=128, dtype=0, starts=A16, ends=A16, mask=A16, words=2,
             out=A16, lse=0, requests=1, R=4, heads=8, scale=1.0, ws=WS, wsb=1 << 40)
    assert set(kw) <= set(a)
    a.update(kw)
    return A._load().mqa_attend_tree(
        cache() if c is None else c, P(a["q"]), a["q_row"], a["q_head"], a["dtype"], P(a["starts"]),
        P(a["ends"]), P(a["mask"]), a["words"], P(a["out"]), P(a["lse"]), a["requests"], a["R"],
        a["heads"], a["scale"], P(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("call", [window, tree])
def test_attention_errors(call):
    for name in ("q", "starts", "ends", "out"):
        assert call(**{name: 0}) == 1, name
    assert call(cache(pages=0)) == 1
    for kw in (dict(q=0x10008), dict(out=MIS), dict(starts=0x10002), dict(lse=0x10002),
               dict(ws=0x20080), dict(q_row=1020), dict(q_head=132)):
        assert call(**kw) == 2, kw
    for kw in (dict(requests=0), dict(R=0), dict(heads=7), dict(dtype=2), dict(scale=-1.0),
               dict(scale=float("nan")), dict(q_row=-1024)):
        assert call(**kw) == 3, kw
    assert call(cache(head_dim=80)) == 3


def test_window_errors():
    for kw in (dict(window=0), dict(window=-1), dict(sinks=-1)):
        assert window(**kw) == 3, kw


def test_tree_errors():
    assert tree(mask=0) == 1
    assert tree(mask=0x10002) == 2
    for kw in (dict(words=0), dict(words=33), dict(words=-1)):
        assert tree(**kw) == 3, kw


def test_no_device_is_an_error_not_a_fallback():
    import torch
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU")
    assert window() == 5
    assert window(window=(1 << 31) - 1, sinks=(1 << 31) - 1) == 5
    assert tree() == 5
    assert rotate() == 5
    assert weigh() == 5
    assert select() == 5
    assert keep() == 5
    assert rotate(k=None, kv_heads=0, rot=0, pos=0, f=0) == 5


H = S._HeadRows


def rotate(**kw):
    a = dict(q=H(A16, 1024, 128), q_out=H(A16, 1024, 128), heads=8, k=H(A16, 256, 128),
             k_out=H(A16, 256, 128), kv_heads=2, qw=A16, kw=A16, wt=0, pos=A16, f=A16, rot=128, pairs=0,
             rows=4, D=128, dtype=0, norm=1, eps=1e-6)
    assert set(kw) <= set(a)
    a.update(kw)
    return S._load().mqa_norm_rotate(a["q"], a["q_out"], a["heads"], a["k"], a["k_out"], a["kv_heads"],
                                     P(a["qw"]), P(a["kw"]), a["wt"], P(a["pos"]), P(a["f"]), a["rot"],
                                     a["pairs"], a["rows"], a["D"], a["dtype"], a["norm"], a["eps"], None)


def test_norm_rotate_errors():
    for name in ("q", "q_out", "k", "k_out"):
        assert rotate(**{name: None}) == 1, name
        assert rotate(**{name: H(0, 1024, 128)}) == 1, name
        assert rotate(**{name: H(0x10008, 1024, 128)}) == 2, name
        assert rotate(**{name: H(A16, 1020, 128)}) == 2, name
        assert rotate(**{name: H(A16, 1024, 4)}) == 2, name
        assert rotate(**{name: H(A16, -1024, 128)}) == 3, name
    assert rotate(pos=0) == 1 and rotate(f=0) == 1
    for kw in (dict(qw=0x10008), dict(kw=0x10008), dict(pos=0x10002), dict(f=0x10004)):
        assert rotate(**kw) == 2, kw
    for kw in (dict(rows=0), dict(rows=(1 << 20) + 1), dict(heads=0), dict(heads=1025), dict(kv_heads=-1),
               dict(kv_heads=1025), dict(D=96), dict(D=512), dict(dtype=2), dict(wt=1), dict(rot=24),
               dict(rot=144), dict(rot=-16), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(q_out=H(A16, 0, 128)), dict(k_out=H(A16, 256, 0))):
        assert rotate(**kw) == 3, kw


def test_exports_match_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mqa_serve.h")).read(), flags=re.S)
    names = set(re.findall(r"^[a-z_][a-z0-9_ ]*[ *]+(\w+)\(", text, flags=re.M))
    assert names == set(mqa.SERVE_EXPORTS)
    for n in names:
        assert hasattr(S._load(), n), n


def test_header_is_c_and_the_structure_is_the_bindings(tmp_path):
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "t.c"
    src.write_text('#include <stdio.h>\n#include "mqa_serve.h"\nint main(void) {'
                   + "".join(f'printf("%zu ", offsetof(mqa_head_rows, {f}));' for f, _ in H._fields_)
                   + 'printf("%zu", sizeof(mqa_head_rows)); return 0; }\n')
    exe = tmp_path / "t"
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                    str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert [int(x) for x in got] == [getattr(H, f).offset for f, _ in H._fields_] + [ctypes.sizeof(H)]


def weigh(c=None, **kw):
    a = dict(q=A16, q_row=1024, q_head=128, dtype=0, starts=A16, ends=A16, lse=A16, weights=A16, width=256,
             requests=1, R=4, heads=8, scale=1.0, ws=WS, wsb=1 << 40)
    assert set(kw) <= set(a)
    a.update(kw)
    return S._load().mqa_kv_weigh(
        cache() if c is None else c, P(a["q"]), a["q_row"], a["q_head"], a["dtype"], P(a["starts"]),
        P(a["ends"]), P(a["lse"]), P(a["weights"]), a["width"], a["requests"], a["R"], a["heads"],
        a["scale"], P(a["ws"]), a["wsb"], None)


def select(**kw):
    a = dict(weights=A16, width=256, lengths=A16, keep=64, sinks=4, recent=16, positions=A16, counts=A16,
             kept=A16, requests=2, ws=WS, wsb=1 << 40)
    assert set(kw) <= set(a)
    a.update(kw)
    return S._load().mqa_kv_select(P(a["weights"]), a["width"], P(a["lengths"]), a["keep"], a["sinks"],
                                   a["recent"], P(a["positions"]), P(a["counts"]), P(a["kept"]),
                                   a["requests"], P(a["ws"]), a["wsb"], None)


def keep(c=None, **kw):
    a = dict(positions=A16, counts=A16, starts=A16, width=64, requests=2, ws=WS, wsb=1 << 40)
    assert set(kw) <= set(a)
    a.update(kw)
    return S._load().mqa_kv_keep(cache() if c is None else c, P(a["positions"]), P(a["counts"]),
                                 P(a["starts"]), a["width"], a["requests"], P(a["ws"]), a["wsb"], None)


def test_weigh_errors():
    for name in ("q", "starts", "ends", "lse", "weights"):
        assert weigh(**{name: 0}) == 1, name
    assert weigh(cache(table=0)) == 1
    for kw in (dict(q=0x10008), dict(starts=0x10002), dict(ends=0x10002), dict(lse=0x10002),
               dict(weights=0x10002), dict(ws=0x20080), dict(q_row=1020), dict(q_head=132)):
        assert weigh(**kw) == 2, kw
    for kw in (dict(width=0), dict(requests=0), dict(R=0), dict(requests=1 << 11, R=1 << 10), dict(heads=7),
               dict(heads=0), dict(heads=1026), dict(dtype=2), dict(scale=-1.0), dict(scale=float("inf")),
               dict(q_row=-1024)):
        assert weigh(**kw) == 3, kw
    assert weigh(cache(block=128)) == 3


def test_select_errors():
    for name in ("weights", "lengths", "positions", "counts"):
        assert select(**{name: 0}) == 1, name
        assert select(**{name: 0x10002}) == 2, name
    assert select(kept=0x10002) == 2
    assert select(ws=0x20080) == 2
    for kw in (dict(width=0), dict(width=(1 << 20) + 1), dict(keep=0), dict(keep=(1 << 20) + 1), dict(sinks=-1),
               dict(recent=-1), dict(sinks=60, recent=5), dict(sinks=(1 << 31) - 1, recent=(1 << 31) - 1),
               dict(requests=0), dict(requests=(1 << 20) + 1), dict(requests=1 << 20, keep=65)):
        assert select(**kw) == 3, kw


def test_keep_errors():
    for name in ("positions", "counts"):
        assert keep(**{name: 0}) == 1, name
    for kw in (dict(positions=0x10002), dict(counts=0x10002), dict(starts=0x10002), dict(ws=0x20080)):
        assert keep(**kw) == 2, kw
    for kw in (dict(width=0), dict(width=(1 << 20) + 1), dict(requests=0), dict(requests=1 << 20, width=65)):
        assert keep(**kw) == 3, kw
    assert keep(cache(head_dim=96)) == 3
    size = S._load().workspace_size_keep
    assert size(1, 5000, 1, 64, 16) >= 2 * 5000 * 64 and size(64, 5000, 8, 64, 16) >= 7 * 5000 * 8 * 64
    assert size(1, 100, 1, 64, 16) == 256
    for bad in ((0, 1, 1, 64, 16), (1, 0, 1, 64, 16), (1, 1, 0, 64, 16), (1, 1, 1, 96, 16), (1, 1, 1, 64, 8),
                (1, 1, 1, 64, 48), (1 << 20, 65, 1, 64, 16)):
        assert size(*bad) == 0, bad
    most = size(16, 4096, 8, 128, 64)
    for n, w in ((16, 4096), (1, 4096), (16, 1), (3, 777)):
        assert 0 < size(n, w, 8, 128, 64) <= most


def test_workspaces_of_selection_serve_smaller_calls():
    size = S._load().workspace_size_select
    for bad in ((0, 1), (1, 0), ((1 << 20) + 1, 1), (1, (1 << 20) + 1)):
        assert size(*bad) == 0, bad
    assert size(1, 4096) == 256 and size(1 << 20, 4096) == 256 and size(1, 20000) > 256
    for requests, width in ((1, 65536), (40, 20000), (600, 1 << 20), (511, 4097)):
        most = size(requests, width)
        for n in (1, 2, 3, 7, 8, 31, 40, 100, 256, 511, 512, 600):
            for w in (1, 4096, 4097, 8192, 20000, 65536, 1 << 20):
                if n <= requests and w <= width:
                    assert size(n, w) <= most
