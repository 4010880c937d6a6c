"""Offsets past 32 bits: caches and inputs larger than 4 GiB give what small ones give."""
import pytest
import torch

import fp8_mqa_logits_amd as mqa
import serve_ref
from gpu_helpers import say
from test_gpu_attend import layout, problem
from test_gpu_evict import lists_of

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def test_pages_far_into_a_large_pool():
    lens = [900, 500]
    pool, table, q, starts, ends = problem(lens, 3, 8, 2, 128, 64, 64, BF16, "e4m3")
    L, small = layout(pool), pool.bytes().cuda()
    pages = (9 << 30) // L.page_bytes
    big = torch.empty(pages, L.page_bytes, dtype=torch.uint8, device="cuda")
    # every page of the small pool somewhere past 4 GiB, every other one past 8
    place = torch.tensor([((4 << 30) if i % 2 else (8 << 30)) // L.page_bytes + 2 + i
                          for i in range(len(small))], device="cuda")
    big[place] = small
    near = table.cuda()
    far = torch.where(near >= 0, place[near.clamp(min=0).long()].int(), near)
    q, s, e = q.cuda(), starts.cuda(), ends.cuda()
    say("case: pages past 4 and 8 GiB")
    both = ((small, near), (big, far))
    win = [mqa.mqa_attend_window(L, q, c, t, s, e, 200, 4) for c, t in both]
    mask = serve_ref.words(torch.eye(3, dtype=torch.bool).repeat(2, 1)).cuda()
    trees = [mqa.mqa_attend_tree(L, q, c, t, s, e - 3, mask, return_lse=True) for c, t in both]
    full = [mqa.mqa_attend_paged(L, q, c, t, s, e, return_lse=True)[1] for c, t in both]
    weights = [mqa.mqa_kv_weigh(L, q, c, t, s, e, full[0], torch.zeros(2, table.shape[1] * 64, device="cuda"))
               for c, t in both]
    assert torch.equal(*win) and torch.equal(trees[0][0], trees[1][0]) and torch.equal(*weights)
    many = q.repeat_interleave(150, 0).contiguous()  # weighed on the wide kernel
    args = [t.repeat_interleave(150, 0).contiguous() for t in (s, e, full[0])]
    weights = [mqa.mqa_kv_weigh(L, many, c, t, *args, torch.zeros(2, table.shape[1] * 64, device="cuda"))
               for c, t in both]
    assert torch.equal(*weights)
    listed, count = lists_of(lens, [0, 0], 0.4, 3)
    kept = [mqa.mqa_kv_read(L, mqa.mqa_kv_keep(L, c, t, listed.cuda(), count.cuda()), t,
                            torch.zeros(2, dtype=torch.int32, device="cuda"), count.cuda(), 900)
            for c, t in both]
    assert torch.equal(kept[0][0], kept[1][0]) and torch.equal(kept[0][1], kept[1][1])


def test_moving_without_room_in_place_far_into_a_large_pool():
    # few heads and a long list: through the workspace
    lens = [5000]
    pool, table, *_ = problem(lens, 1, 2, 2, 64, 64, 16, BF16, "int8")
    L, small = layout(pool), pool.bytes().cuda()
    assert mqa.workspace_size_keep(1, 2000, L) > 256
    first = (5 << 30) // L.page_bytes
    big = torch.empty(first + len(small), L.page_bytes, dtype=torch.uint8, device="cuda")
    big[first:] = small
    near = table.cuda()
    far = torch.where(near >= 0, near + first, near)
    listed, count = (t.cuda() for t in lists_of(lens, [0], 0.4, 3))
    mqa.mqa_kv_keep(L, small, near, listed, count)
    mqa.mqa_kv_keep(L, big, far, listed, count)
    assert torch.equal(big[first:], small)


def test_rows_far_apart():
    # three rows, the last ones past 2^31 and 2^32 elements
    far = torch.empty((1 << 32) + 4096, dtype=BF16, device="cuda")
    x = torch.as_strided(far, (3, 6, 128), (1 << 31, 128, 1))
    g = torch.Generator().manual_seed(2)
    x.copy_(torch.randn(3, 6, 128, generator=g).to(BF16))
    w = torch.ones(128, dtype=BF16, device="cuda")
    f = (10000.0 ** (-torch.arange(0, 128, 2) / 128)).float().cuda()
    pos = torch.tensor([5, 6, 7]).int().cuda()
    near = x.contiguous()
    want = mqa.mqa_norm_rotate(near[:, :4], near[:, 4:], w, w, pos, f)
    got = mqa.mqa_norm_rotate(x[:, :4], x[:, 4:], w, w, pos, f, q_out=x[:, :4], k_out=x[:, 4:])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("requests,width", [(3, 300000), (1, 1 << 20), (600, 20000)])
def test_selection_of_long_rows(requests, width):
    g = torch.Generator(device="cuda")
    g.manual_seed(width)
    w = torch.rand(requests, width, generator=g, device="cuda")
    w[:, ::3] = 0.5  # many equal weights, some of them at the border
    length = torch.full((requests,), width, dtype=torch.int32, device="cuda")
    length[-1] = width // 2
    keep, sinks, recent = width // 2 - 100, 4, 1000
    listed, count = mqa.mqa_kv_select(w, length, keep, sinks, recent)
    at = torch.arange(width, device="cuda")
    rank = torch.where((at < sinks) | (at >= length[:, None] - recent), 2.0, w)
    rank = torch.where(at < length[:, None], rank, -1.0)
    best = rank.sort(dim=1, descending=True, stable=True).indices[:, :keep].sort(dim=1).values
    assert count.tolist() == [keep] * requests
    assert torch.equal(listed.long(), best)
