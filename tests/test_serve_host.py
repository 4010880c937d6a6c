"""Host-side checks of what a serving step does around attention: bad arguments are
refused before any device memory is touched. No GPU needed (nothing here launches
work; the addresses are never used)."""
import ctypes

import pytest

from fp8_mqa_logits_amd import attend as A
from test_attend_host import A16, MIS, WS, cache

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
