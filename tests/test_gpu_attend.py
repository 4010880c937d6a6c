"""Attention over the paged 8-bit cache against the 64-bit reference: ranges
and lists, both code types, head layouts, odd lengths, and what unseen
positions may hold. Tolerances: attend_ref.attend."""
import math

import pytest
import torch

import attend_ref as ref
import fp8_mqa_logits_amd as mqa
from gpu_helpers import say

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


def problem(lens, R, Hq, Hkv, D, P, B, dtype, codes, see="causal", seed=1, extra=1):
    table, pages = ref.make_table(lens, P, seed, extra=extra)
    pool = ref.Pool(pages, Hkv, D, P, B, codes, seed)
    g = torch.Generator().manual_seed(seed + 1)
    # scores of a few units: k is up to 8 * 2^2 a channel
    q = (torch.randn(len(lens) * R, Hq, D, generator=g) * 0.15).to(dtype)
    t = torch.arange(R).repeat(len(lens))
    length = torch.tensor(lens).repeat_interleave(R)
    ends, starts = length - (R - 1 - t), torch.zeros(len(lens) * R, dtype=torch.long)
    if see == "window":
        starts = ends - 37
    if see == "full":
        ends = length
    if see == "mixed":  # empty, past the end, negative, reversed, single positions
        for i in range(len(starts)):
            starts[i], ends[i] = [(0, 0), (5, length[i] + 1000), (-7, 3), (9, 2), (11, 12),
                                  (int(length[i]) // 2, int(length[i]))][i % 6]
        ends = torch.minimum(ends, length)
        ends[1::6] = length[1::6]
    return pool, table, q, starts.int(), ends.int()


def layout(pool):
    Hkv, D, P, B = pool.dims
    return mqa.KVLayout(Hkv, D, P, B, pool.kind)


def reached(pool, table, ends):
    """The table without the pages past every row's end."""
    return table[:, :max(1, -(-int(ends.max()) // pool.dims[2]))]


def check(pool, table, q, starts, ends, indices=None, scale=None):
    want, lse, tol, tol_lse = ref.attend(pool, q, reached(pool, table, ends), starts, ends, scale,
                                         indices)
    args = [layout(pool), q.cuda(), pool.bytes().cuda(), table.cuda()]
    if indices is not None:
        args.append(indices.cuda())
    call = mqa.mqa_attend_paged if indices is None else mqa.mqa_attend_topk
    out, got_lse = call(*args, starts.cuda(), ends.cuda(), scale=scale, return_lse=True)
    torch.cuda.synchronize()
    assert out.dtype == q.dtype and out.shape == q.shape
    assert ref.differs(out, want, tol) == 0
    assert ref.differs(got_lse, lse, tol_lse) == 0
    return out, got_lse


SHAPES = [
    # lens, R, Hq, Hkv, D, P, B
    ([1], 1, 1, 1, 64, 16, 16),
    ([1], 1, 8, 8, 128, 64, 64),
    ([15, 16, 17], 1, 8, 2, 128, 16, 16),
    ([63, 64, 65, 1], 1, 5, 1, 64, 64, 16),
    ([700, 3, 129, 128], 1, 32, 8, 128, 64, 32),
    ([300, 41], 4, 10, 2, 64, 32, 32),
    ([333, 90], 7, 12, 12, 128, 128, 64),
    ([1500], 3, 64, 1, 128, 64, 64),
    ([600], 1, 128, 1, 128, 32, 16),
    ([257], 2, 96, 2, 64, 16, 16),
    ([260], 40, 16, 2, 128, 64, 64),
    ([515], 130, 8, 2, 64, 32, 16),
    ([400], 333, 4, 4, 128, 64, 32),
    ([333], 70, 28, 4, 128, 128, 128),
    ([2100, 2049], 1, 16, 2, 128, 256, 64),
    ([40000], 1, 8, 2, 128, 64, 64),
]


@pytest.mark.parametrize("dtype,codes", [(BF16, "e4m3"), (FP16, "int8"), (FP16, "e4m3"),
                                         (BF16, "int8")])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[1:])))
def test_ranges(shape, dtype, codes):
    for see in ("causal", "window") if shape[1] > 1 else ("causal",):
        say(f"case: attend_paged {shape} {dtype} {codes} {see}")
        check(*problem(*shape, dtype, codes, see))


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[1] in (4, 7, 40, 130)],
                         ids=lambda s: "x".join(map(str, s[1:])))
@pytest.mark.parametrize("see", ["mixed", "full"])
def test_rows_of_any_range(shape, see):
    say(f"case: attend_paged {shape} {see}")
    out, lse = check(*problem(*shape, BF16, "e4m3", see))
    if see == "mixed":
        assert bool((out[0::6] == 0).all()) and bool((lse[0::6] == -math.inf).all())
        assert bool((out[3::6] == 0).all()) and bool((lse[3::6] == -math.inf).all())


# calls whose tables have room for 131072 positions run on tiles of 128 and 256
# columns however short their contexts are
CHUNKS = [s for s in SHAPES if s[1] in (40, 70, 130, 333)] + [
    ([700, 90], 20, 8, 2, 128, 64, 64),
    ([70], 17, 8, 2, 64, 16, 16),
    ([3000], 70, 4, 1, 64, 64, 32),
]


@pytest.mark.parametrize("dtype,codes", [(BF16, "e4m3"), (FP16, "int8"), (FP16, "e4m3"),
                                         (BF16, "int8")])
@pytest.mark.parametrize("shape", CHUNKS, ids=lambda s: "x".join(map(str, s[1:])))
def test_wide_tiles(shape, dtype, codes):
    for see in ("causal", "window", "full", "mixed"):
        say(f"case: wide tiles {shape} {dtype} {codes} {see}")
        check(*problem(*shape, dtype, codes, see, extra=131072 // shape[5]))


@pytest.mark.parametrize("dtype,codes,D", [(BF16, "e4m3", 128), (FP16, "int8", 128),
                                           (FP16, "e4m3", 64), (BF16, "int8", 64)])
@pytest.mark.parametrize("R", [20, 45])
@pytest.mark.parametrize("loud", [1.0, 6.0])
def test_wide_tiles_over_many_keys(R, loud, dtype, codes, D):
    # requests enough for one part each, so that every workgroup goes through
    # dozens of tiles; with loud scores the rows' largest ones are met all along
    say(f"case: many keys {R} {loud} {dtype} {codes} {D}")
    lens, times = [2300, 1111, 1984], 44
    pool, table, q, starts, ends = problem(lens, R, 8, 2, D, 64, 32, dtype, codes)
    q = (q.float() * loud).to(dtype)
    want, lse, tol, tol_lse = ref.attend(pool, q, table, starts, ends)
    out, got_lse = mqa.mqa_attend_paged(
        layout(pool), q.cuda().repeat(times, 1, 1), pool.bytes().cuda(),
        table.cuda().repeat(times, 1), starts.cuda().repeat(times), ends.cuda().repeat(times),
        return_lse=True)
    assert ref.differs(out, want.repeat(times, 1, 1), tol.repeat(times, 1, 1)) == 0
    assert ref.differs(got_lse, lse.repeat(times, 1), tol_lse.repeat(times, 1)) == 0


@pytest.mark.parametrize("split", [97, 128])
def test_packed_requests(split):
    # two requests in one key numbering, each row with its own request's range
    say(f"case: packed {split}")
    pool, table, q, starts, ends = problem([700], 260, 8, 2, 128, 64, 64, BF16, "e4m3")
    starts[split:] = 320
    ends[:split] = 320 - split + 1 + torch.arange(split)
    check(pool, table, q, starts, ends)


def lists(starts, ends, width, seed, padding=0.2):
    """Distinct positions of each row's range in any order, -1 anywhere."""
    g = torch.Generator().manual_seed(seed)
    out = torch.full((len(starts), width), -1, dtype=torch.int32)
    for r in range(len(starts)):
        n = max(0, int(ends[r]) - max(0, int(starts[r])))
        at = torch.randperm(n, generator=g)[:width].int()
        at[torch.rand(len(at), generator=g) < padding] = -1
        out[r, :len(at)] = at
    return out


@pytest.mark.parametrize("dtype,codes", [(BF16, "e4m3"), (FP16, "int8"), (FP16, "e4m3"),
                                         (BF16, "int8")])
@pytest.mark.parametrize("shape,width", [
    (SHAPES[0], 1), (SHAPES[2], 8), (SHAPES[3], 33), (SHAPES[4], 64), (SHAPES[5], 100),
    (SHAPES[7], 512), (SHAPES[8], 333), (SHAPES[9], 47), (SHAPES[11], 128), (SHAPES[14], 2048),
    (SHAPES[15], 5000)], ids=lambda s: "x".join(map(str, s[1:])) if isinstance(s, tuple) else str(s))
def test_lists(shape, width, dtype, codes):
    say(f"case: attend_topk {shape} {width} {dtype} {codes}")
    p = problem(*shape, dtype, codes, "window" if shape[1] == 4 else "causal")
    check(*p, indices=lists(p[3], p[4], width, 5))


def test_list_entries_outside_the_range_and_twice():
    say("case: attend_topk, entries outside and twice")
    pool, table, q, starts, ends = problem([300, 200], 2, 8, 2, 128, 32, 32, BF16, "e4m3", "window")
    idx = lists(starts, ends, 40, 3)
    idx[0, :4] = torch.tensor([5, 5, 5, 36])     # 36: the last, then past the end
    idx[1, :3] = torch.tensor([37, 1 << 30, -5])
    idx[2] = -1                                  # a row that lists nothing
    check(pool, table, q, starts, ends, indices=idx)


def test_list_of_everything_is_the_range():
    say("case: list of everything")
    pool, table, q, starts, ends = problem([500, 310], 3, 16, 4, 128, 64, 64, BF16, "e4m3")
    idx = torch.arange(512).int().repeat(6, 1)
    a, la = check(pool, table, q, starts, ends, indices=idx)
    b, lb = check(pool, table, q, starts, ends)
    assert torch.allclose(la, lb, atol=1e-5)


@pytest.mark.parametrize("room", [1, 4096])  # (pages past the contexts: wider tiles)
@pytest.mark.parametrize("R,Hq", [(1, 8), (5, 8), (90, 8), (3, 64), (200, 32)])
@pytest.mark.parametrize("codes", ["e4m3", "int8"])
def test_unseen_positions_may_hold_anything(R, Hq, codes, room):
    # NaN codes and NaN, infinite and negative scales in slots no row sees
    say(f"case: garbage {R} {Hq} {codes}")
    lens = [411, 250]
    pool, table, q, starts, ends = problem(lens, R, Hq, 2, 128, 32, 16, BF16, codes, "causal",
                                           extra=room)
    starts += 100
    clean = pool.bytes()
    args = (starts.cuda(), ends.cuda())
    a, want_lse = mqa.mqa_attend_paged(layout(pool), q.cuda(), clean.cuda(), table.cuda(), *args,
                                       return_lse=True)
    used = torch.zeros(pool.codes.shape[0], 32, dtype=torch.bool)
    for i, n in enumerate(lens):
        pos = torch.arange(100, n)
        used[table[i].long()[pos // 32], pos % 32] = True
    pool.codes[~used.view(-1, 1, 1, 32, 1).expand_as(pool.codes)] = 0x7F if codes == "e4m3" else 0x80
    blocks = used.view(-1, 2, 16).any(-1)
    n = int((~blocks).sum()) * 4
    bad = torch.tensor([math.nan, math.inf, -1.0]).repeat(n // 3 + 1)[:n]
    pool.scales[~blocks.view(-1, 1, 1, 2).expand_as(pool.scales)] = bad
    b, lse = mqa.mqa_attend_paged(layout(pool), q.cuda(), pool.bytes().cuda(), table.cuda(), *args,
                                  return_lse=True)
    assert torch.equal(a, b) and torch.equal(want_lse, lse) and bool((lse < math.inf).all())
    idx = lists(starts, ends, 64, 8)
    clean_out = mqa.mqa_attend_topk(layout(pool), q.cuda(), clean.cuda(), table.cuda(), idx.cuda(), *args)
    out = mqa.mqa_attend_topk(layout(pool), q.cuda(), pool.bytes().cuda(), table.cuda(), idx.cuda(), *args)
    assert torch.equal(clean_out, out)


@pytest.mark.parametrize("room", [1, 4096])  # (pages past the contexts: wider tiles)
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("R,Hq", [(4, 8), (40, 8), (150, 16)])
def test_nan_reaches_only_the_rows_that_see_it(R, Hq, where, room):
    say(f"case: NaN in {where}, {R} rows")
    pool, table, q, starts, ends = problem([400], R, Hq, 2, 128, 32, 32, BF16, "e4m3", "causal",
                                           extra=room)
    at = 400 - R // 2  # the later rows see it
    pool.codes[table[0, at // 32].long(), 0 if where == "k" else 1, 1, at % 32, 5] = 0x7F
    out = mqa.mqa_attend_paged(layout(pool), q.cuda(), pool.bytes().cuda(), table.cuda(),
                               starts.cuda(), ends.cuda()).float().cpu()
    sees = ends > at
    heads = torch.arange(Hq) >= Hq // 2
    assert 0 < int(sees.sum()) < R
    assert bool(torch.isfinite(out[~sees]).all()) and bool(torch.isfinite(out[:, ~heads]).all())
    hit = torch.isnan(out[sees][:, heads])
    assert bool(hit.all()) if where == "k" else bool(hit[..., 5].all())
    want, _, tol, _ = ref.attend(pool, q, reached(pool, table, ends), starts, ends)
    assert ref.differs(out[~sees], want[~sees], tol[~sees]) == 0


@pytest.mark.parametrize("R", [1, 12, 70])
def test_nan_of_a_position_without_weight(R):
    # the first half of the keys, scored 5000 below the others, holds a NaN value
    say(f"case: NaN without weight, {R} rows")
    pool, table, q, starts, ends = problem([20000], R, 8, 1, 128, 64, 64, BF16, "e4m3", "full")
    first = table[0, :156].long()
    pool.codes[first, 0] = 0xFE
    pool.scales[first, 0] = 1.0
    pool.codes[first[7], 1, 0, 9, 5] = 0x7F
    q = torch.ones_like(q)
    starts[1::2] = 12000  # does not see it
    for idx in (None, torch.arange(20000).int().repeat(R, 1)):
        args = [layout(pool), q.cuda(), pool.bytes().cuda(), table.cuda()]
        args += [] if idx is None else [idx.cuda()]
        call = mqa.mqa_attend_paged if idx is None else mqa.mqa_attend_topk
        out = call(*args, starts.cuda(), ends.cuda()).float().cpu()
        assert bool(torch.isnan(out[0::2, :, 5]).all()) and bool(torch.isfinite(out[1::2]).all())


@pytest.mark.parametrize("R,room", [(1, 1), (40, 1), (100, 1), (40, 8192), (100, 8192)])
def test_scales_of_very_different_size(R, room):
    # value scales that fall and rise by 2^40 along the context, zero blocks
    # among them; the softmax sees all of them
    say(f"case: uneven scales, {R} rows")
    pool, table, q, starts, ends = problem([640], R, 8, 2, 128, 32, 16, BF16, "e4m3", "causal",
                                           extra=room)
    for j in range(40):
        page, b = int(table[0, j * 16 // 32]), j * 16 % 32 // 16
        pool.scales[page, 1, :, b] = [2.0 ** -20, 1.0, 0.0, 2.0 ** 20, 2.0 ** -8][j % 5]
        if j % 7 == 3:
            pool.scales[page, 0, :, b] = 0.0
    check(pool, table, q, starts, ends)
    low = pool.scales[:, 1] * 2.0 ** -100
    pool.scales[:, 1] = low
    check(pool, table, q, starts, ends)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("R,room", [(1, 1), (30, 1), (30, 4096), (70, 4096)])
def test_one_appended_token_is_what_read_gives(R, room, dtype):
    # a row that sees one position has probability 1, and append's scales are
    # powers of two: the very value that a read returns
    say(f"case: single appended keys, {R} rows {dtype}")
    L = mqa.KVLayout(kv_heads=2, head_dim=128, page_size=32, block=16, codes="e4m3")
    table = torch.full((1, 7 + room), -1, dtype=torch.int32)
    table[0, :7] = torch.randperm(7, generator=torch.Generator().manual_seed(3)).int()
    cache = torch.zeros(7, L.page_bytes, dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(200, 2, 128, generator=g).to(dtype).cuda() for _ in range(2))
    first = torch.zeros(1, dtype=torch.int32, device="cuda")
    mqa.mqa_kv_append(L, k, v, cache, table.cuda(), first)
    starts = torch.arange(R).int() + 50
    q = torch.randn(R, 8, 128, generator=g).to(dtype).cuda()
    _, want = mqa.mqa_kv_read(L, cache, table.cuda(), first + 50, None, R, dtype=dtype)
    want = want.repeat_interleave(4, dim=1)
    out = mqa.mqa_attend_paged(L, q, cache, table.cuda(), starts.cuda(), (starts + 1).cuda())
    assert torch.equal(out, want)
    idx = torch.full((R, 8), -1, dtype=torch.int32)
    idx[:, 3] = 0
    out = mqa.mqa_attend_topk(L, q, cache, table.cuda(), idx.cuda(), starts.cuda(),
                              (starts + 1).cuda())
    assert torch.equal(out, want)


def test_one_small_block_decides():
    # a row whose softmax lies in a block 2^30 below its neighbours' scale
    say("case: small block decides")
    pool, table, q, starts, ends = problem([128], 20, 4, 1, 64, 64, 16, FP16, "e4m3", "full")
    pool.scales[:] = 1.0 / 64
    pool.scales[int(table[0, 0]), 1, 0, 0] = 2.0 ** -24
    pool.codes[int(table[0, 0]), 0, 0, :16] = 0x7E  # loud keys
    q = q.abs() + 1.0
    check(pool, table, q.half(), starts, ends)


@pytest.mark.parametrize("scale", [0.0, 0.01, 3.0])
@pytest.mark.parametrize("R", [1, 90])
def test_score_scale(scale, R):
    say(f"case: scale {scale}, {R} rows")
    check(*problem([300], R, 8, 2, 64, 32, 32, BF16, "e4m3"), scale=scale)


def test_large_scores_do_not_overflow():
    say("case: large scores")
    pool, table, q, starts, ends = problem([300], 90, 8, 2, 128, 32, 32, BF16, "e4m3")
    check(pool, table, (q.float() * 300).to(BF16), starts, ends)


@pytest.mark.parametrize("R", [1, 3, 90])
def test_strides(R):
    # q a slice of a wider projection, pages of several layers interleaved
    say(f"case: strides, {R} rows")
    pool, table, q, starts, ends = problem([300, 77], R, 8, 2, 128, 32, 32, BF16, "e4m3")
    want, lse, tol, _ = ref.attend(pool, q, table, starts, ends)
    wide = torch.full((2 * R, 12, 136), 7.0, dtype=BF16, device="cuda")
    wide[:, 2:10, 8:] = q.cuda()
    layers = torch.full((pool.codes.shape[0], 3, pool.bytes().shape[1]), 0x7F, dtype=torch.uint8,
                        device="cuda")
    layers[:, 1] = pool.bytes().cuda()
    got = mqa.mqa_attend_paged(layout(pool), wide[:, 2:10, 8:], layers[:, 1], table.cuda(),
                               starts.cuda(), ends.cuda())
    assert ref.differs(got, want, tol) == 0
    swapped = q.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    got = mqa.mqa_attend_paged(layout(pool), swapped, layers[:, 1], table.cuda(), starts.cuda(),
                               ends.cuda())
    assert ref.differs(got, want, tol) == 0


def test_pages_past_four_gibibytes():
    say("case: pages past 4 GiB")
    pool, table, q, starts, ends = problem([200], 3, 8, 2, 128, 64, 64, BF16, "e4m3")
    want, _, tol, _ = ref.attend(pool, q, table, starts, ends)
    n, size = pool.codes.shape[0], pool.bytes().shape[1]
    far = (5 << 30) // size
    cache = torch.empty(far + n, size, dtype=torch.uint8, device="cuda")
    cache[far:] = pool.bytes().cuda()
    moved = torch.where(table >= 0, table + far, table)
    for call, more in ((mqa.mqa_attend_paged, ()),
                       (mqa.mqa_attend_topk, (torch.arange(256).int().repeat(3, 1).cuda(),))):
        got = call(layout(pool), q.cuda(), cache, moved.cuda(), *more, starts.cuda(), ends.cuda())
        assert ref.differs(got, want, tol) == 0


@pytest.mark.parametrize("shape", [SHAPES[4], SHAPES[11], SHAPES[15]])
def test_same_bits_again_and_on_another_stream(shape):
    say(f"case: again {shape}")
    pool, table, q, starts, ends = problem(*shape, BF16, "e4m3")
    args = [layout(pool), q.cuda(), pool.bytes().cuda(), table.cuda(), starts.cuda(), ends.cuda()]
    a, la = mqa.mqa_attend_paged(*args, return_lse=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [mqa.mqa_attend_paged(*args, return_lse=True, stream=s) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(s)
    for b, lb in outs:
        assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("shape", [SHAPES[4], SHAPES[11]])
def test_graph_replays(shape):
    say(f"case: graph {shape}")
    pool, table, q, starts, ends = problem(*shape, BF16, "e4m3")
    L, qd, cache = layout(pool), q.cuda(), pool.bytes().cuda()
    idx = lists(starts, ends, 64, 4).cuda()
    more = (table.cuda(), starts.cuda(), ends.cuda())
    n = mqa.workspace_size_attend(len(table), shape[1], shape[2], L, table.shape[1] * shape[5])
    work = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty_like(qd) for _ in range(2)]

    def both():
        mqa.mqa_attend_paged(L, qd, cache, *more, out=outs[0], workspace=work[0])
        mqa.mqa_attend_topk(L, qd, cache, more[0], idx, *more[1:], out=outs[1], workspace=work[1])

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for k in range(4):
        qd.copy_((q.float() * (1 + 0.3 * k)).to(BF16))
        both()
        want = [o.clone() for o in outs]
        torch.cuda.synchronize()
        for o in outs:
            o.zero_()
        for w in work:
            w.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_workspace_holds_anything_before():
    say("case: dirty workspace")
    pool, table, q, starts, ends = problem([3000, 10], 2, 16, 2, 128, 64, 64, BF16, "e4m3")
    L = layout(pool)
    n = mqa.workspace_size_attend(2, 2, 16, L, table.shape[1] * 64)
    outs = []
    for fill in (0, 0xFF, 0x7F):
        w = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        outs.append(mqa.mqa_attend_paged(L, q.cuda(), pool.bytes().cuda(), table.cuda(),
                                         starts.cuda(), ends.cuda(), workspace=w))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_binding_refusals():
    pool, table, q, starts, ends = problem([100], 2, 8, 2, 128, 32, 32, BF16, "e4m3")
    L, cache = layout(pool), pool.bytes().cuda()
    q, table, starts, ends = q.cuda(), table.cuda(), starts.cuda(), ends.cuda()
    call = mqa.mqa_attend_paged
    with pytest.raises(TypeError):
        call(L, q.float(), cache, table, starts, ends)
    with pytest.raises(ValueError):
        call(L, q[:, :, :64], cache, table, starts, ends)
    with pytest.raises(ValueError):
        call(L, q.cpu(), cache, table, starts, ends)
    with pytest.raises(ValueError):
        call(L, q, cache[:, :-16], table, starts, ends)
    with pytest.raises(TypeError):
        call(L, q, cache, table, starts.long(), ends)
    with pytest.raises(ValueError):
        call(L, q, cache, table, starts[:1], ends)
    with pytest.raises(ValueError):
        call(L, q, cache, table, starts, ends, out=torch.empty_like(q)[:, :4])
    with pytest.raises(mqa.MQAError) as e:
        call(L, q[:, :7], cache, table, starts, ends)
    assert e.value.code == 3
    with pytest.raises(mqa.MQAError) as e:
        call(L, q, cache, table, starts, ends, scale=-1.0)
    assert e.value.code == 3
    many = torch.zeros(1, 2000, dtype=torch.int32, device="cuda")  # keys in parts
    size = mqa.workspace_size_attend(1, 2, 8, L, 2000 * 32)
    assert size > 256
    for n, code in ((0, 1), (512, 4)):
        with pytest.raises(mqa.MQAError) as e:
            call(L, q, cache, many, starts, ends,
                 workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
        assert e.value.code == code
    wide = torch.zeros(2, 8, 132, dtype=BF16, device="cuda")
    with pytest.raises(mqa.MQAError) as e:
        call(L, wide[:, :, 4:], cache, table, starts, ends)
    assert e.value.code == 2
    with pytest.raises(ValueError):
        mqa.mqa_attend_topk(L, q, cache, table, torch.zeros(3, 4, dtype=torch.int32, device="cuda"),
                            starts, ends)
    with pytest.raises(TypeError):
        mqa.mqa_attend_topk(L, q, cache, table, None, starts, ends)


def test_strides_of_axes_of_one_element_do_not_matter():
    # one row of a projection whose width is no multiple of 8, one key head
    say("case: strides of single rows and heads")
    pool, table, q, starts, ends = problem([300], 1, 8, 1, 128, 32, 32, BF16, "e4m3")
    want, _, tol, _ = ref.attend(pool, q, table, starts, ends)
    args = (pool.bytes().cuda(), table.cuda(), starts.cuda(), ends.cuda())
    row = torch.empty(3 * 1037, dtype=BF16, device="cuda").as_strided((1, 8, 128), (1037, 128, 1))
    row.copy_(q)
    assert ref.differs(mqa.mqa_attend_paged(layout(pool), row, *args), want, tol) == 0
    L, cache = layout(pool), args[0]
    k = torch.empty(4000, dtype=BF16, device="cuda").as_strided((1, 1, 128), (1037, 131, 1))
    k.copy_(torch.randn(1, 1, 128))
    at = torch.tensor([299], dtype=torch.int32, device="cuda")
    mqa.mqa_kv_append(L, k, k, cache, args[1], at)
    got, _ = mqa.mqa_kv_read(L, cache, args[1], at, None, 1)
    assert float((got - k).abs().max()) <= 2.0 ** -4 * float(k.abs().max())
