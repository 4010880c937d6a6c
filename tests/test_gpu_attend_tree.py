"""Attention over trees of drafted tokens against the 64-bit reference: trees,
chains and arbitrary masks, contexts that end anywhere, both kinds of tiles.
Tolerances: serve_ref.attend."""
import math

import pytest
import torch

import attend_ref as ref
import fp8_mqa_logits_amd as mqa
import serve_ref
from gpu_helpers import say
from test_gpu_attend import layout, problem

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


def trees(N, R, seed, spread=8):
    """[N * R, R] bool: a draft sees itself and its ancestors; parents are up to
    `spread` drafts back (1: a chain)."""
    g = torch.Generator().manual_seed(seed)
    back = torch.randint(1, spread + 1, (N, R), generator=g)
    see = torch.zeros(N, R, R, dtype=torch.bool)
    for i in range(N):
        for t in range(R):
            parent = t - int(back[i, t])
            if parent >= 0:
                see[i, t] = see[i, parent]
            see[i, t, t] = True
    return see.view(N * R, R)


def check(pool, table, q, starts, ends, bits, scale=None):
    cap = table.shape[1] * pool.dims[2]
    mask = serve_ref.words(bits)
    seen = serve_ref.tree_seen(starts, ends, mask, cap)
    want, lse, tol, tol_lse = serve_ref.attend(pool, q, table, seen[:, :max(1, int(seen.any(0).nonzero().max()) + 1)] if seen.any() else seen[:, :1], scale)
    out, got_lse = mqa.mqa_attend_tree(layout(pool), q.cuda(), pool.bytes().cuda(), table.cuda(),
                                       starts.cuda(), ends.cuda(), mask.cuda(), scale=scale,
                                       return_lse=True)
    torch.cuda.synchronize()
    assert ref.differs(out, want, tol) == 0
    assert ref.differs(got_lse, lse, tol_lse) == 0
    return out, got_lse


SHAPES = [
    # lens (drafts included), R, Hq, Hkv, D, P, B
    ([2, 33], 2, 1, 1, 64, 16, 16),
    ([700, 13, 129, 128], 5, 32, 8, 128, 64, 32),
    ([300, 41], 31, 10, 2, 64, 32, 32),
    ([333, 90], 33, 12, 12, 128, 128, 64),
    ([1500], 64, 64, 1, 128, 16, 16),
    ([515], 130, 8, 2, 64, 32, 16),
    ([40000], 3, 8, 2, 128, 64, 64),
]


def drafted(shape, dtype, codes, extra=1):
    pool, table, q, starts, _ = problem(*shape, dtype, codes, extra=extra)
    R = shape[1]
    ends = torch.tensor([n - R for n in shape[0]]).repeat_interleave(R).int()
    return pool, table, q, starts, ends


@pytest.mark.parametrize("dtype,codes", [(BF16, "e4m3"), (FP16, "int8"), (FP16, "e4m3"), (BF16, "int8")])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[1:])))
def test_trees(shape, dtype, codes):
    say(f"case: attend_tree {shape} {dtype} {codes}")
    check(*drafted(shape, dtype, codes), trees(len(shape[0]), shape[1], 3))


@pytest.mark.parametrize("dtype,codes", [(BF16, "e4m3"), (FP16, "int8")])
@pytest.mark.parametrize("shape", [s for s in SHAPES if 2 < s[1] and max(s[0]) < 2000],
                         ids=lambda s: "x".join(map(str, s[1:])))
def test_wide_tiles(shape, dtype, codes):
    # (a table with room for 131072 positions runs on the widest tile for its columns)
    say(f"case: wide tree {shape} {dtype} {codes}")
    check(*drafted(shape, dtype, codes, extra=131072 // shape[5]), trees(len(shape[0]), shape[1], 4))


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[1] in (5, 31, 64, 130)],
                         ids=lambda s: "x".join(map(str, s[1:])))
@pytest.mark.parametrize("wide", [False, True])
def test_any_ranges_and_masks(shape, wide):
    # rows of empty, reversed and clamped ranges, masks of random bits, of none and of
    # bits past the table's end; rows of one request that end at different positions
    say(f"case: tree mixed {shape} {wide}")
    pool, table, q, starts, ends = problem(*shape, BF16, "e4m3", "mixed",
                                           extra=131072 // shape[5] if wide else 1)
    g = torch.Generator().manual_seed(9)
    rows = len(starts)
    bits = torch.rand(rows, 100, generator=g) < 0.3
    bits[::7] = False
    bits[3::5, 32:64] = False
    # drafts lie in pages that the table names
    length = torch.tensor(shape[0]).repeat_interleave(shape[1])
    last = -(-length // pool.dims[2]) * pool.dims[2]
    e = serve_ref.ranges(starts, ends, table.shape[1] * pool.dims[2])[1]
    bits &= (e + torch.arange(100) < last[:, None])
    out, lse = check(pool, table, q, starts, ends, bits)
    none = ((starts.clamp(min=0) >= ends) & ~bits.any(1)).nonzero()[:, 0]
    assert len(none) and bool((out[none] == 0).all()) and bool((lse[none] == -math.inf).all())


def test_bits_past_the_table_name_nothing():
    pool, table, q, starts, ends = drafted(([64], 8, 4, 2, 64, 16, 16), BF16, "e4m3", extra=0)
    full = torch.ones(8, 1024, dtype=torch.bool)
    out, _ = check(pool, table, q, starts, ends, full)
    some = full.clone()
    some[:, 8:] = False
    assert torch.equal(out, check(pool, table, q, starts, ends, some)[0])


def test_what_no_row_sees_may_be_anything():
    # NaN codes at drafts that no row sees, and at one that a single row sees
    shape = ([300], 24, 8, 2, 128, 64, 16)
    for extra in (1, 4096):
        pool, table, q, starts, ends = drafted(shape, BF16, "e4m3", extra)
        bits = trees(1, 24, 6)
        bits[:, 11] = False
        bits[:, 17] = False
        bits[20, 17] = True
        for x in (11, 17):
            at = 300 - 24 + x
            pool.codes[int(table[0, at // 64]), 1, :, at % 64] = 0x7F
        say(f"case: tree with NaN drafts, extra {extra}")
        out, _ = check(pool, table, q, starts, ends, bits)
        bad = torch.isnan(out.float()).any(2).any(1)
        assert bad.nonzero()[:, 0].tolist() == [20]


@pytest.mark.parametrize("extra", [1, 4096])
def test_a_chain_is_a_causal_range(extra):
    # the same positions under another description; sums in the same order
    shape = ([500, 77], 20, 8, 2, 128, 64, 64)
    pool, table, q, starts, ends = drafted(shape, BF16, "e4m3", extra)
    chain = trees(2, 20, 1, spread=1)
    args = [layout(pool), q.cuda(), pool.bytes().cuda(), table.cuda(), starts.cuda()]
    t = torch.arange(20).repeat(2).int()
    got = mqa.mqa_attend_tree(*args, ends.cuda(), serve_ref.words(chain).cuda())
    want = mqa.mqa_attend_paged(*args, (ends + t + 1).cuda())
    tol = (2 * 2.0 ** -8 + 2.0 ** -9) * want.float().abs().amax()
    assert float((got.float() - want.float()).abs().max()) <= tol


def test_refusals():
    pool, table, q, starts, ends = drafted(([64], 8, 4, 2, 64, 16, 16), BF16, "e4m3")
    args = [layout(pool), q.cuda(), pool.bytes().cuda(), table.cuda(), starts.cuda(), ends.cuda()]
    good = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        mqa.mqa_attend_tree(*args, None)
    with pytest.raises(TypeError):
        mqa.mqa_attend_tree(*args, good.long())
    for bad in (good[:4], good[:, 0], good.cpu(), torch.zeros(8, 4, dtype=torch.int32, device="cuda")[:, ::2]):
        with pytest.raises(ValueError):
            mqa.mqa_attend_tree(*args, bad)
    for words in (0, 33):
        with pytest.raises(mqa.MQAError):
            mqa.mqa_attend_tree(*args, torch.zeros(8, words, dtype=torch.int32, device="cuda"))
