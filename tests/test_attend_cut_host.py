"""How attention calls are cut into tiles and parts, as the host decides it. No GPU needed."""
import ctypes

import pytest

from fp8_mqa_logits_amd import attend as A

CUS = 256
RANGES, LISTS, WINDOWS, TREES = range(4)


def cut(kind, requests, R, heads, kv_heads, head_dim, positions, window=0, sinks=0, cus=CUS):
    """(columns a tile, tiles, parts)"""
    out = (ctypes.c_int32 * 3)()
    assert A._load().mqa_attend_cut(kind, requests, R, heads, kv_heads, head_dim, positions, window,
                                    sinks, cus, out) == 0
    return tuple(out)


@pytest.mark.parametrize("R,window,columns", [(16384, 8192, 256), (16384, 4096, 256), (8192, 8192, 256),
                                              (8192, 2048, 32), (4096, 4096, 32)])
def test_prompts_that_fill_their_table(R, window, columns):
    # what was measured to be the fastest (12 heads, each its own key head): the table's
    # room bounds the call, but not what a row sees
    assert cut(WINDOWS, 1, R, 12, 12, 128, R, window, 4)[::2] == (columns, 1)


def test_a_window_is_not_told_by_the_room_that_bounds_it():
    plans = {cut(WINDOWS, 1, 8192, 12, 12, 128, 8192, window, 0) for window in (30, 2000, 8000)}
    assert len(plans) > 1


@pytest.mark.parametrize("R", [1, 5, 64, 700, 4096])
@pytest.mark.parametrize("heads,kv_heads,head_dim", [(32, 8, 128), (12, 12, 64), (16, 4, 128), (64, 1, 64)])
def test_windows_do_not_depend_on_room_that_they_do_not_reach(heads, kv_heads, head_dim, R):
    for window, sinks in ((1, 0), (500, 4), (2000, 70)):
        rows = 256 // (heads // kv_heads) + 1  # of the widest tile
        least = window + sinks + min(rows, R) + 1
        plans = {cut(WINDOWS, 3, R, heads, kv_heads, head_dim, max(least, room), window, sinks)
                 for room in (least, R, 2 * R + least, 1 << 20, (1 << 31) - 1)}
        assert len(plans) == 1, (window, sinks)


def test_tiles_hold_all_columns():
    for kind in (RANGES, WINDOWS, TREES):
        for R, heads, kv_heads in ((1, 1, 1), (13, 40, 8), (130, 8, 2), (4096, 32, 4), (1 << 20, 8, 8)):
            for room in (16, 777, 131072, (1 << 31) - 1):
                columns, tiles, parts = cut(kind, 1, R, heads, kv_heads, 128, room, 1000, 4)
                assert columns in (16, 32, 64, 128, 256) and 1 <= parts <= 256
                assert (tiles - 1) * columns < R * (heads // kv_heads) <= tiles * columns
    assert cut(LISTS, 3, 4, 32, 8, 128, 2048)[1] == 1
    assert cut(WINDOWS, 1, 1, 8, 8, 64, 1 << 20, (1 << 31) - 1, (1 << 31) - 1)[2] >= 1


def test_windows_and_trees_are_planned_on_tiles_that_are_built():
    # no kernels of 64 columns, nor of 256 for heads of 64
    for kind in (WINDOWS, TREES):
        for head_dim, built in ((64, {16, 32, 128}), (128, {16, 32, 128, 256})):
            seen = set()
            for heads, kv_heads in ((1, 1), (8, 2), (32, 8), (12, 12), (64, 1), (1024, 1), (1024, 1024)):
                for requests in (1, 3, 30, 300):
                    for R in (1, 5, 17, 40, 64, 333, 2000):
                        for room in (16, 1000, 9000, 131072, 1 << 20):
                            for window in (1, 300, 5000, 1 << 20) if kind == WINDOWS else (1,):
                                seen.add(cut(kind, requests, R, heads, kv_heads, head_dim, room, window, 4)[0])
            assert seen == built


def test_errors():
    call = A._load().mqa_attend_cut
    out = (ctypes.c_int32 * 3)(7, 7, 7)
    good = dict(kind=2, requests=1, R=4, heads=8, kv_heads=2, head_dim=64, positions=100, window=1, sinks=0,
                cus=CUS)
    assert call(*good.values(), None) == 1
    for kw in (dict(kind=-1), dict(kind=4), dict(requests=0), dict(R=0), dict(requests=1 << 11, R=1 << 10),
               dict(heads=7), dict(heads=1026), dict(kv_heads=0), dict(head_dim=96), dict(positions=0),
               dict(window=0), dict(window=-5), dict(sinks=-1), dict(cus=0)):
        assert call(*{**good, **kw}.values(), out) == 3, kw
    assert tuple(out) == (7, 7, 7)
    assert call(*{**good, "kind": 0, "window": 0}.values(), out) == 0
