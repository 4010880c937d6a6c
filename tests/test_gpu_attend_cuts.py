"""Windows with sinks and trees of drafts on every wide tile that they are planned on:
tiles of 128 and 256 columns, whole and in parts, with pages between sinks and windows in
other use and drafts that hold NaN, against the 64-bit reference. Which tile a call runs on
is asked for, not assumed. Tolerances: serve_ref.attend."""
import ctypes
import math

import pytest
import torch

import attend_ref as ref
import fp8_mqa_logits_amd as mqa
import serve_ref
from fp8_mqa_logits_amd import attend as A
from gpu_helpers import say
from test_gpu_attend import layout, problem
from test_gpu_attend_tree import trees

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16
BOTH = [(BF16, "e4m3"), (FP16, "int8"), (FP16, "e4m3"), (BF16, "int8")]


def cut_of(kind, requests, R, Hq, Hkv, D, room, window=0, sinks=0):
    """(columns a tile, whether keys are cut into parts)"""
    out = (ctypes.c_int32 * 3)()
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert A._load().mqa_attend_cut(kind, requests, R, Hq, Hkv, D, room, window, sinks, cus, out) == 0
    return out[0], out[2] > 1


def repeated(times, q, table, starts, ends):
    return (q.cuda().repeat(times, 1, 1), table.cuda().repeat(times, 1), starts.cuda().repeat(times),
            ends.cuda().repeat(times))


def compare(out, lse, times, want, wlse, tol, tol_lse):
    """The first requests against the reference, the repeated ones bit for bit against them.
    A row and head that sees a value's NaN code is NaN in its column at least."""
    out, lse = out.view(times, *want.shape), lse.view(times, *wlse.shape)
    first, bad = out[0].cpu(), torch.isnan(want)
    assert bool(torch.isnan(first[bad]).all())
    ill = bad.any(2, keepdim=True)
    assert ref.differs(torch.where(ill, 0.0, first), torch.where(ill, 0.0, want), tol.nan_to_num(0.0)) == 0
    assert ref.differs(lse[0], wlse, tol_lse) == 0
    bits = out.view(torch.int16)
    assert bool((bits == bits[0]).all()) and bool((lse == lse[0]).all())


WINDOWS = [
    # lens, R, Hq, Hkv, D, P, B; times, window, sinks; columns, parts
    (([700, 431, 590], 64, 8, 2, 64, 16, 16), 40, 150, 4, 128, False),
    (([900, 431], 64, 16, 2, 64, 64, 32), 50, 300, 70, 128, False),
    (([3300, 2900, 2703], 40, 16, 1, 64, 64, 64), 10, 2500, 70, 128, True),
    (([2900, 2711], 40, 16, 1, 128, 32, 16), 45, 2500, 17, 128, False),
    (([6500, 6301, 6400], 40, 16, 1, 128, 64, 64), 10, 6000, 100, 128, True),
    (([700, 433, 590], 64, 16, 1, 128, 16, 16), 20, 300, 20, 256, False),
    (([1200, 1111], 64, 16, 2, 128, 128, 64), 30, 700, 4, 256, False),
    (([4500, 4201, 4400], 64, 16, 2, 128, 64, 32), 10, 4000, 65, 256, True),
]


def window_id(c):
    return f"{'x'.join(map(str, c[0][1:]))}-{c[2]}+{c[3]}-{c[4]}{'-parts' if c[5] else ''}"


@pytest.mark.parametrize("dtype,codes", BOTH)
@pytest.mark.parametrize("case", WINDOWS, ids=window_id)
@pytest.mark.parametrize("freed", [False, True])
def test_windows(case, dtype, codes, freed):
    shape, times, window, sinks, columns, parts = case
    lens, R, Hq, Hkv, D, P, B = shape
    say(f"case: cut windows {case} {dtype} {codes} {freed}")
    pool, table, q, starts, ends = problem(*shape, dtype, codes)
    room = table.shape[1] * P
    assert cut_of(2, len(lens) * times, R, Hq, Hkv, D, room, window, sinks) == (columns, parts)
    # sinks stand apart from the windows, more than a step of 64 away
    assert min(lens[0], room) - R - window > sinks + 128
    seen = serve_ref.window_seen(starts, ends, window, sinks, room)
    want, wlse, tol, tol_lse = serve_ref.attend(pool, q, table, seen)
    if freed:
        spoilt = set(range(pool.codes.shape[0]))
        named = table.clone()
        for i in range(len(lens)):
            used = seen[i * R:(i + 1) * R].any(0).view(-1, P).any(1)
            spoilt -= set(named[i][used].tolist())
            junk = torch.tensor([-1, 1 << 30, -(1 << 31), sorted(spoilt)[0]], dtype=torch.int32)
            table[i] = torch.where(used, named[i], junk[torch.arange(table.shape[1]) % 4])
        for i in range(len(lens)):  # (a page that stands for nothing in one may serve another)
            spoilt -= set(named[i][seen[i * R:(i + 1) * R].any(0).view(-1, P).any(1)].tolist())
        spoilt = torch.tensor(sorted(spoilt))
        assert len(spoilt)
        pool.codes[spoilt] = 0x7F
        pool.scales[spoilt] = math.nan
        pool.scales[spoilt[::2]] = math.inf
    if codes == "e4m3":  # a value in the sinks of all rows and one in the first row's window only
        at = int(ends[0]) - window
        pool.codes[int(table[0, 0]), 1, 0, 0, 5] = 0x7F
        pool.codes[int(table[0, at // P]), 1, Hkv - 1, at % P, 9] = 0x7F
        want, wlse, tol, tol_lse = serve_ref.attend(pool, q, table.clamp(0, len(pool.codes) - 1), seen)
        first = torch.isnan(want[0]).any(1)
        assert bool(first[0]) and bool(first[-1])
    args = repeated(times, q, table, starts, ends)
    out, lse = mqa.mqa_attend_window(layout(pool), args[0], pool.bytes().cuda(), *args[1:], window, sinks,
                                     return_lse=True)
    compare(out, lse, times, want, wlse, tol, tol_lse)


TREES = [
    # lens (drafts included), R, Hq, Hkv, D, P, B; times, room; columns, parts
    (([700, 431, 590], 70, 8, 2, 64, 16, 16), 60, 1024, 128, False),
    (([1900, 1431], 64, 16, 2, 64, 64, 32), 6, 8192, 128, True),
    (([700, 931], 40, 16, 1, 128, 32, 16), 45, 1024, 128, False),
    (([1500, 931], 40, 16, 1, 128, 64, 64), 15, 8192, 128, True),
    (([700, 433, 590], 64, 16, 1, 128, 16, 16), 20, 1024, 256, False),
    (([1500, 2111], 64, 16, 1, 128, 128, 64), 10, 8192, 256, True),
]


@pytest.mark.parametrize("dtype,codes", BOTH)
@pytest.mark.parametrize("case", TREES, ids=lambda c: f"{'x'.join(map(str, c[0][1:]))}-{c[3]}{'-parts' if c[4] else ''}")
@pytest.mark.parametrize("masks", ["trees", "any"])
def test_trees(case, dtype, codes, masks):
    shape, times, room, columns, parts = case
    lens, R, Hq, Hkv, D, P, B = shape
    say(f"case: cut trees {case} {dtype} {codes} {masks}")
    extra = room // P - -(-max(lens) // P)
    pool, table, q, starts, _ = problem(*shape, dtype, codes, extra=extra)
    assert table.shape[1] * P == room
    assert cut_of(3, len(lens) * times, R, Hq, Hkv, D, room) == (columns, parts)
    ends = torch.tensor([n - R for n in lens]).repeat_interleave(R).int()
    bits = trees(len(lens), R, 3)
    if masks == "any":  # bits of any draft; rows without any, and without a range
        bits = torch.rand(bits.shape, generator=torch.Generator().manual_seed(4)) < 0.4
        bits[::7] = False
        starts[::5] = ends[::5]
    # a draft that no row sees, and one that a single row does, hold NaN
    bits[:, 11 % R] = False
    bits[:, 7] = False
    bits[5, 7] = True
    if codes == "e4m3":
        for i, x in ((0, 11 % R), (0, 7), (1, 11 % R)):
            at = lens[i] - R + x
            pool.codes[int(table[i, at // P]), 1, :, at % P] = 0x7F
    mask = serve_ref.words(bits)
    seen = serve_ref.tree_seen(starts, ends, mask, max(lens))
    want, wlse, tol, tol_lse = serve_ref.attend(pool, q, table, seen)
    if codes == "e4m3":
        assert torch.isnan(want).any(2).any(1).nonzero()[:, 0].tolist() == [5]
    args = repeated(times, q, table, starts, ends)
    out, lse = mqa.mqa_attend_tree(layout(pool), args[0], pool.bytes().cuda(), *args[1:],
                                   mask.cuda().repeat(times, 1), return_lse=True)
    compare(out, lse, times, want, wlse, tol, tol_lse)
    if masks == "any":
        assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all())


@pytest.mark.parametrize("shape,window,sinks", [(([20000, 9000], 1, 16, 2, 128, 64, 64), 8000, 4),
                                                (([30000], 2, 8, 1, 64, 64, 64), 12345, 300),
                                                (([2600], 2, 64, 1, 128, 64, 64), 2500, 4)],
                         ids=lambda s: "x".join(map(str, s[1:])) if isinstance(s, tuple) else str(s))
def test_few_rows_are_in_parts(shape, window, sinks):
    pool, table, q, starts, ends = problem(*shape, BF16, "e4m3")
    lens, R, Hq, Hkv, D, P, B = shape
    room = table.shape[1] * P
    columns, parts = cut_of(2, len(lens), R, Hq, Hkv, D, room, window, sinks)
    say(f"case: windows in parts {shape} {columns}")
    assert parts
    seen = serve_ref.window_seen(starts, ends, window, sinks, room)
    want, wlse, tol, tol_lse = serve_ref.attend(pool, q, table, seen)
    out, lse = mqa.mqa_attend_window(layout(pool), q.cuda(), pool.bytes().cuda(), table.cuda(), starts.cuda(),
                                     ends.cuda(), window, sinks, return_lse=True)
    assert ref.differs(out, want, tol) == 0 and ref.differs(lse, wlse, tol_lse) == 0
