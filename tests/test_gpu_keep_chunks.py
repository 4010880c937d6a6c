"""Moving in place, in more than one round: lists of more tokens than a workgroup holds at
once, of requests and heads enough to need no workspace, against reading and storing again."""
import pytest
import torch

import attend_ref as ref
import fp8_mqa_logits_amd as mqa
from fp8_mqa_logits_amd import attend as A
from fp8_mqa_logits_amd import serve as S
from gpu_helpers import say
from test_gpu_attend import layout
from test_gpu_evict import check_keep, lists_of

pytestmark = pytest.mark.gpu

SHAPES = [
    # lens, Hkv, D, P, B
    ([4100, 2600, 1400, 1050], 16, 64, 64, 16), ([3900, 1025, 2048, 2700], 16, 128, 64, 32),
    ([2300, 4000], 32, 64, 128, 64), ([2500, 1100, 30, 3300, 1024, 0, 2049, 1], 8, 128, 16, 16),
    ([3333], 64, 128, 64, 64)]


def pool_of(shape, codes, seed, nan_codes=False):
    lens, Hkv, D, P, B = shape
    table, pages = ref.make_table(lens, P, seed)
    return table, ref.Pool(pages, Hkv, D, P, B, codes, seed, nan_codes=nan_codes)


def in_place(pool, table, listed):
    """Whether a call of these sizes needs no workspace (one of empty lists, without any)."""
    cache, d = pool.bytes().cuda(), table.cuda()
    c, dev, requests = A._cache(layout(pool), cache, d)
    none = torch.zeros(requests, dtype=torch.int32, device="cuda")
    rc = S._load().mqa_kv_keep(c, listed.cuda().data_ptr(), none.data_ptr(), None, listed.shape[1], requests,
                               None, 0, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc in (0, 1)
    return listed.shape[1] > 1024 and rc == 0


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[1:])))
@pytest.mark.parametrize("share", [0.97, 0.999, 0.6])
def test_moving(shape, codes, share):
    # dense lists: sources right behind their places, over the borders of rounds
    say(f"case: keep in rounds {shape} {codes} {share}")
    table, pool = pool_of(shape, codes, 1, nan_codes=share == 0.6)
    listed, counts = lists_of(shape[0], [0] * len(shape[0]), share, 3)
    assert in_place(pool, table, listed)
    check_keep(pool, table, listed, counts)


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[1:])))
def test_moving_behind_what_stays(shape, codes):
    # starts inside blocks, each another; counts that end inside blocks
    lens = shape[0]
    starts = [min(n, (37 * i + 5) % 200) for i, n in enumerate(lens)]
    for share in (0.98, 0.7):
        say(f"case: keep in rounds behind {shape} {codes} {share}")
        table, pool = pool_of(shape, codes, 2)
        listed, counts = lists_of(lens, starts, share, 4)
        assert in_place(pool, table, listed)
        counts -= torch.arange(len(lens)).int() % 3
        check_keep(pool, table, listed, counts, torch.tensor(starts).int())


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("back", [0, 21])
def test_positions_named_twice_and_entries_that_name_none(codes, back):
    shape = SHAPES[1]
    say(f"case: keep in rounds, any entries {codes} {back}")
    table, pool = pool_of(shape, codes, 5)
    g = torch.Generator().manual_seed(6)
    lens, width = shape[0], 2500
    counts = torch.tensor([2500, 1000, 1500, 2100]).int()
    listed = torch.full((4, width), -1, dtype=torch.int32)
    for i, (n, c) in enumerate(zip(lens, counts.tolist())):
        # entry t names back + t or a position behind it, up to the last; ascending
        x = back + torch.arange(c) + torch.randint(0, 40, (c,), generator=g)
        x = torch.maximum(x.sort().values, back + torch.arange(c)).clamp(max=n - 1)
        assert bool((x >= back + torch.arange(c)).all()) and bool((x.diff() == 0).any())
        listed[i, :c] = x.int()
        none = torch.rand(c, generator=g) < 0.1
        listed[i, :c][none] = torch.where(torch.rand(int(none.sum()), generator=g) < 0.5, -1, 1 << 20).int()
    assert in_place(pool, table, listed)
    check_keep(pool, table, listed, counts, torch.full((4,), back).int())


def test_replays_and_another_stream():
    shape = SHAPES[2]
    table, pool = pool_of(shape, "e4m3", 7)
    L, d = layout(pool), table.cuda()
    listed, counts = (t.cuda() for t in lists_of(shape[0], [0, 0], 0.9, 8))
    fresh, cache = pool.bytes().cuda(), pool.bytes().cuda()
    want = mqa.mqa_kv_keep(L, fresh.clone(), d, listed, counts)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mqa.mqa_kv_keep(L, cache, d, listed, counts)
    for _ in range(3):
        cache.copy_(fresh)
        graph.replay()
        assert torch.equal(cache, want)
    side = torch.cuda.Stream()
    cache.copy_(fresh)
    torch.cuda.synchronize()
    mqa.mqa_kv_keep(L, cache, d, listed, counts, stream=side)
    side.synchronize()
    assert torch.equal(cache, want)
