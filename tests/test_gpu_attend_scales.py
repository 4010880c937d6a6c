"""Attention over the paged 8-bit cache where value scales differ widely: blocks
that no row sees, rows beside louder rows, and rows whose softmax lies in quiet
blocks. Reference and tolerances: attend_ref.attend (scales here are large enough
that its absolute term of 2^-25 has no part)."""
import math

import pytest
import torch

import attend_ref as ref
import fp8_mqa_logits_amd as mqa
from gpu_helpers import say
from test_gpu_attend import layout, lists, problem

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16

# rows and query heads (of 2 key heads) that make tiles of 16, 32, 64, 128 and 256
# columns where the table has room for long contexts; without room all take 16
TILES = [(2, 8), (4, 16), (6, 16), (8, 32), (20, 32)]
LENGTH, P, B = 700, 32, 16


def garbage_gap(pool, table, gap, scale, codes, entries):
    """The cache and table with `scale` and the largest codes in the blocks of
    positions [gap[0], gap[1]); entries: of the pages that lie in it whole, "own" or
    "none" (-1, which reads as page 0)."""
    g = ref.Pool(len(pool.codes) + 1, *pool.dims, pool.kind, 1)
    g.codes[1:], g.scales[1:] = pool.codes, pool.scales
    g.codes[0] = 0x7E if codes == "e4m3" else 0x80
    g.scales[0] = scale
    moved = torch.where(table >= 0, table + 1, table)
    for pos in range(gap[0], gap[1], B):
        page, b = int(moved[0, pos // P]), pos % P // B
        g.codes[page, :, :, pos % P:pos % P + B] = 0x7E if codes == "e4m3" else 0x80
        g.scales[page, :, :, b] = scale
    if entries == "none":
        moved[0, -(-gap[0] // P):gap[1] // P] = -1
    return g, moved


@pytest.mark.parametrize("codes,dtype", [("e4m3", BF16), ("int8", FP16)])
@pytest.mark.parametrize("room", [1, 4096])
@pytest.mark.parametrize("R,Hq", TILES)
def test_blocks_between_the_rows_ranges_may_hold_anything(R, Hq, room, codes, dtype):
    # two packed requests, and windows apart, with whole blocks between them
    # that no row sees: the same bits whatever those hold
    pool, table, q, starts, ends = problem([LENGTH], R, Hq, 2, 128, P, B, dtype, codes, "full",
                                           extra=room)
    first = torch.arange(R) < R // 2
    for see, gap in (("packed", (208, 416)), ("apart", (48, 640))):
        if see == "packed":
            starts = torch.where(first, 0, 421).int()
            ends = torch.where(first, 202 - torch.arange(R), LENGTH).int()
        else:
            starts = torch.where(torch.arange(R) % 2 == 0, 645, 3).int()
            ends = (starts + 40).int()
        args = (starts.cuda(), ends.cuda())
        want, want_lse = mqa.mqa_attend_paged(layout(pool), q.cuda(), pool.bytes().cuda(),
                                              table.cuda(), *args, return_lse=True)
        exact, exact_lse, tol, tol_lse = ref.attend(pool, q, table[:, :-(-LENGTH // P)], starts, ends)
        assert ref.differs(want, exact, tol) == 0 and ref.differs(want_lse, exact_lse, tol_lse) == 0
        for scale in (2.0 ** 20, 1e12, 1e30, 3e38, math.inf, math.nan):
            for entries in ("own", "none"):
                say(f"case: gap {R} {Hq} {room} {codes} {see} {scale} {entries}")
                g, moved = garbage_gap(pool, table, gap, scale, codes, entries)
                out, lse = mqa.mqa_attend_paged(layout(g), q.cuda(), g.bytes().cuda(),
                                                moved.cuda(), *args, return_lse=True)
                assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("first,codes", [("quiet", "e4m3"), ("loud", "int8")])
@pytest.mark.parametrize("apart", [12, 30, 60])
@pytest.mark.parametrize("room", [1, 4096])
@pytest.mark.parametrize("R,Hq", TILES)
def test_rows_beside_louder_rows(R, Hq, room, codes, apart, first):
    # two packed requests in a tile, the values of one 2^apart times the other's
    say(f"case: beside louder rows {R} {Hq} {room} {codes} {apart} {first}")
    pool, table, q, starts, ends = problem([LENGTH], R, Hq, 2, 128, P, B, BF16, codes, "full",
                                           extra=room)
    for pos in range(0, LENGTH, B):
        if (pos < 320) == (first == "loud"):
            pool.scales[int(table[0, pos // P]), 1, :, pos % P // B] *= 2.0 ** apart
    early = torch.arange(R) < R // 2
    starts, ends = torch.where(early, 0, 320).int(), torch.where(early, 320, LENGTH).int()
    want, lse, tol, tol_lse = ref.attend(pool, q, table[:, :-(-LENGTH // P)], starts, ends)
    out, got_lse = mqa.mqa_attend_paged(layout(pool), q.cuda(), pool.bytes().cuda(), table.cuda(),
                                        starts.cuda(), ends.cuda(), return_lse=True)
    assert ref.differs(out, want, tol) == 0
    assert ref.differs(got_lse, lse, tol_lse) == 0


def quiet_weight(pool, table, loud, ratio):
    """Blocks of the positions in `loud` get keys of the lowest code (scores far
    below the others' for positive queries) and values 2^ratio louder."""
    for pos in loud:
        page, b = int(table[0, pos // P]), pos % P // B
        pool.codes[page, 0, :, pos % P:pos % P + B] = 0xFE if pool.kind == "e4m3" else 0x81
        pool.scales[page, 0, :, b] = 1.0 / 64 if pool.kind == "e4m3" else 1.0 / 18
        pool.scales[page, 1, :, b] *= 2.0 ** ratio


@pytest.mark.parametrize("where", ["before", "after", "between"])
@pytest.mark.parametrize("ratio,codes", [(30, "e4m3"), (60, "e4m3"), (34, "int8")])
@pytest.mark.parametrize("room", [1, 4096])
@pytest.mark.parametrize("R,Hq", [(1, 8)] + TILES)
def test_softmax_in_quiet_blocks(R, Hq, room, codes, ratio, where):
    # every row sees blocks 2^ratio louder than those that hold its softmax
    say(f"case: quiet blocks {R} {Hq} {room} {codes} {ratio} {where}")
    pool, table, q, starts, ends = problem([LENGTH], R, Hq, 2, 128, P, B, BF16, codes, "full",
                                           extra=room)
    every = range(0, LENGTH, B)
    loud = {"before": every[:22], "after": every[22:], "between": every[1::2]}[where]
    quiet_weight(pool, table, loud, ratio)
    q = (q.float().abs() + 1.0).to(BF16)
    for p in set(every) - set(loud):  # scores of the others around 0
        pool.scales[int(table[0, p // P]), 0, :, p % P // B] *= 2.0 ** -8
    L, exact_table = layout(pool), table[:, :-(-LENGTH // P)]
    want, lse, tol, tol_lse = ref.attend(pool, q, exact_table, starts, ends)
    out, got_lse = mqa.mqa_attend_paged(L, q.cuda(), pool.bytes().cuda(), table.cuda(),
                                        starts.cuda(), ends.cuda(), return_lse=True)
    assert ref.differs(out, want, tol) == 0
    assert ref.differs(got_lse, lse, tol_lse) == 0
    idx = lists(starts, ends, 512, 7)
    want, lse, tol, tol_lse = ref.attend(pool, q, exact_table, starts, ends, indices=idx)
    out, got_lse = mqa.mqa_attend_topk(L, q.cuda(), pool.bytes().cuda(), table.cuda(), idx.cuda(),
                                       starts.cuda(), ends.cuda(), return_lse=True)
    assert ref.differs(out, want, tol) == 0
    assert ref.differs(got_lse, lse, tol_lse) == 0


@pytest.mark.parametrize("ratio", [20, 26, 40])
@pytest.mark.parametrize("tile", [0, 2])
@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("R,Hq", [(8, 32), (20, 32), (40, 8)])
def test_louder_tile_without_weight_after_a_tile_with_all_of_it(R, Hq, codes, tile, ratio):
    # 64 keys of equal score hold the softmax; all others score far lower, and the
    # next 64 have much larger scales: both halves of the 64 keep their weight
    say(f"case: louder tile after {R} {Hq} {codes} {tile} {ratio}")
    pool, table, q, starts, ends = problem([LENGTH], R, Hq, 2, 128, P, B, BF16, codes, "full",
                                           extra=4096)
    pool.scales[:, 1] = 0.125
    quiet_weight(pool, table, range(0, LENGTH, B), 0)
    for pos in range(64 * tile, 64 * tile + 64):
        pool.codes[int(table[0, pos // P]), 0, :, pos % P] = 0
    for pos in range(64 * tile + 64, 64 * tile + 128, B):
        pool.scales[int(table[0, pos // P]), 1, :, pos % P // B] *= 2.0 ** ratio
    q = (q.float().abs() + 1.0).to(BF16)
    want, lse, tol, tol_lse = ref.attend(pool, q, table[:, :-(-LENGTH // P)], starts, ends)
    out, got_lse = mqa.mqa_attend_paged(layout(pool), q.cuda(), pool.bytes().cuda(), table.cuda(),
                                        starts.cuda(), ends.cuda(), return_lse=True)
    assert ref.differs(out, want, tol) == 0
    assert ref.differs(got_lse, lse, tol_lse) == 0


@pytest.mark.parametrize("where", ["first", "last"])
@pytest.mark.parametrize("codes,silent", [("e4m3", 0.0), ("int8", 2.0 ** -126)])
@pytest.mark.parametrize("room", [1, 4096])
@pytest.mark.parametrize("R,Hq", [(1, 8)] + TILES)
def test_blocks_without_values_count_in_the_softmax(R, Hq, room, codes, silent, where):
    # half of the blocks have value scales of 0, or the least that append writes
    say(f"case: silent blocks {R} {Hq} {room} {codes} {where}")
    pool, table, q, starts, ends = problem([LENGTH], R, Hq, 2, 128, P, B, BF16, codes, "full",
                                           extra=room)
    for pos in range(0, LENGTH, B):
        if (pos < 352) == (where == "first"):
            pool.scales[int(table[0, pos // P]), 1, :, pos % P // B] = silent
    exact_table = table[:, :-(-LENGTH // P)]
    for idx in (None, lists(starts, ends, 512, 7)):
        want, lse, tol, tol_lse = ref.attend(pool, q, exact_table, starts, ends, indices=idx)
        args = [layout(pool), q.cuda(), pool.bytes().cuda(), table.cuda()]
        args += [] if idx is None else [idx.cuda()]
        call = mqa.mqa_attend_paged if idx is None else mqa.mqa_attend_topk
        out, got_lse = call(*args, starts.cuda(), ends.cuda(), return_lse=True)
        assert ref.differs(out, want, tol) == 0
        assert ref.differs(got_lse, lse, tol_lse) == 0


@pytest.mark.parametrize("power", [-88, -60, 50, 94])
@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("room", [1, 4096])
@pytest.mark.parametrize("R,Hq", [(1, 8)] + TILES)
def test_value_scales_of_any_size(R, Hq, room, codes, power):
    # all values 2^power times as large: outputs too, at the same precision
    say(f"case: value scales of 2^{power} {R} {Hq} {room} {codes}")
    pool, table, q, starts, ends = problem([LENGTH], R, Hq, 2, 128, P, B, BF16, codes, extra=room)
    exact_table = table[:, :-(-LENGTH // P)]
    for idx in (None, lists(starts, ends, 512, 7)):
        want, lse, tol, tol_lse = ref.attend(pool, q, exact_table, starts, ends, indices=idx)
        big = ref.Pool(len(pool.codes), *pool.dims, codes, 1)
        big.codes, big.scales = pool.codes, pool.scales.clone()
        big.scales[:, 1] *= 2.0 ** power
        args = [layout(big), q.cuda(), big.bytes().cuda(), table.cuda()]
        args += [] if idx is None else [idx.cuda()]
        call = mqa.mqa_attend_paged if idx is None else mqa.mqa_attend_topk
        out, got_lse = call(*args, starts.cuda(), ends.cuda(), return_lse=True)
        assert ref.differs(out.double() * 2.0 ** -power, want, tol) == 0
        # (e lies 2^power off its usual place: 2^-24 of the exponent more in lse)
        assert ref.differs(got_lse, lse, tol_lse + abs(power) * 2.0 ** -23) == 0
