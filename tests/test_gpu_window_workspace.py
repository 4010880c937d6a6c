"""Workspaces of windows: what a call needs goes by its window and the table's room."""
import pytest
import torch

import fp8_mqa_logits_amd as mqa
from fp8_mqa_logits_amd import attend as A
from test_gpu_attend import layout, problem

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("heads,kv_heads,head_dim", [(32, 8, 128), (12, 12, 64), (64, 1, 128)])
def test_workspaces_of_windows(heads, kv_heads, head_dim):
    # what is needed depends on the window and the room; what serves any window of a span,
    # and what serves the largest batch, are no less
    lib = A._load()
    for requests, R in ((1, 1), (7, 3), (1, 700), (64, 16)):
        largest = lib.workspace_size_attend(requests, R, heads, kv_heads, head_dim, 1 << 20, 0)
        for room in (64, 777, 9000, 131072, 1 << 20):
            for window, sinks in ((1, 0), (500, 4), (8000, 70), (1 << 20, 0), ((1 << 31) - 1, (1 << 31) - 1)):
                need = lib.workspace_size_attend_window(requests, R, heads, kv_heads, head_dim, room, window,
                                                        sinks, 0)
                span = min(window + sinks + R - 1, room)
                any_window = lib.workspace_size_attend_call(requests, R, heads, kv_heads, head_dim, span, 2, 0)
                assert 256 <= need <= any_window <= largest, (requests, R, room, window, sinks)
    good = [2, 3, heads, kv_heads, head_dim, 777, 100, 4, 0]
    assert lib.workspace_size_attend_window(*good) >= 256
    for i, bad in ((0, 0), (1, 0), (2, 0), (4, 80), (5, 0), (6, 0), (7, -1)):
        assert lib.workspace_size_attend_window(*good[:i], bad, *good[i + 1:]) == 0


def test_a_workspace_of_exactly_one_window_s_size():
    pool, table, q, starts, ends = problem([9000], 1, 16, 2, 128, 64, 64, BF16, "e4m3")
    L, lib = layout(pool), A._load()
    n = lib.workspace_size_attend_window(1, 1, 16, 2, 128, table.shape[1] * 64, 8000, 4, 0)
    assert n > 256
    args = (L, q.cuda(), pool.bytes().cuda(), table.cuda(), starts.cuda(), ends.cuda(), 8000, 4)
    want = mqa.mqa_attend_window(*args)
    work = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert torch.equal(mqa.mqa_attend_window(*args, workspace=work), want)
    with pytest.raises(mqa.MQAError):
        mqa.mqa_attend_window(*args, workspace=work[:-256])
