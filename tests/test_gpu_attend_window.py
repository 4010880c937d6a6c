"""Attention through a sliding window with sinks against the 64-bit reference:
windows and sinks of any size and where they meet, rows of any range, what the
positions between them may hold, both kinds of tiles. Tolerances:
serve_ref.attend."""
import math

import pytest
import torch

import attend_ref as ref
import fp8_mqa_logits_amd as mqa
import serve_ref
from fp8_mqa_logits_amd import attend as A
from gpu_helpers import say
from test_gpu_attend import layout, problem

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


def check(pool, table, q, starts, ends, window, sinks, scale=None, want_table=None):
    cap = max(1, min(table.shape[1] * pool.dims[2], int(ends.max()) + pool.dims[2]))
    seen = serve_ref.window_seen(starts, ends, window, sinks, cap)
    want, lse, tol, tol_lse = serve_ref.attend(pool, q, table if want_table is None else want_table,
                                               seen, scale)
    out, got_lse = mqa.mqa_attend_window(layout(pool), q.cuda(), pool.bytes().cuda(), table.cuda(),
                                         starts.cuda(), ends.cuda(), window, sinks, scale=scale,
                                         return_lse=True)
    torch.cuda.synchronize()
    assert out.dtype == q.dtype and out.shape == q.shape
    assert ref.differs(out, want, tol) == 0
    assert ref.differs(got_lse, lse, tol_lse) == 0
    return out, got_lse


SHAPES = [
    # lens, R, Hq, Hkv, D, P, B
    ([1], 1, 1, 1, 64, 16, 16),
    ([700, 3, 129, 128], 1, 32, 8, 128, 64, 32),
    ([300, 41], 4, 10, 2, 64, 32, 32),
    ([333, 90], 7, 12, 12, 128, 128, 64),
    ([1500], 3, 64, 1, 128, 16, 16),
    ([260], 40, 16, 2, 128, 64, 64),
    ([515], 130, 8, 2, 64, 32, 16),
]


@pytest.mark.parametrize("dtype,codes", [(BF16, "e4m3"), (FP16, "int8")])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[1:])))
def test_windows(shape, dtype, codes):
    for window, sinks in ((1, 0), (1, 1), (16, 4), (37, 33), (100, 64), (250, 3), (5, 1000),
                          (1 << 30, 1 << 30)):
        say(f"case: attend_window {shape} {dtype} {codes} window {window} sinks {sinks}")
        check(*problem(*shape, dtype, codes), window, sinks)


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[1] > 1], ids=lambda s: "x".join(map(str, s[1:])))
@pytest.mark.parametrize("window,sinks", [(1, 1), (29, 4), (100, 20)])
def test_rows_of_any_range(shape, window, sinks):
    say(f"case: attend_window mixed {shape} {window} {sinks}")
    out, lse = check(*problem(*shape, BF16, "e4m3", "mixed"), window, sinks)
    assert bool((out[0::6] == 0).all()) and bool((lse[0::6] == -math.inf).all())


# tables with room for 131072 positions and windows past it: tiles of 128 and 256 columns
@pytest.mark.parametrize("dtype,codes", [(BF16, "e4m3"), (FP16, "int8"), (FP16, "e4m3"), (BF16, "int8")])
@pytest.mark.parametrize("shape", [([700, 90], 20, 8, 2, 128, 64, 64), ([515], 130, 8, 2, 64, 32, 16),
                                   ([70], 17, 8, 2, 64, 16, 16), ([333], 70, 28, 4, 128, 128, 128)],
                         ids=lambda s: "x".join(map(str, s[1:])))
def test_wide_tiles_everything_seen(shape, dtype, codes):
    for see in ("causal", "mixed"):
        say(f"case: wide window {shape} {dtype} {codes} {see}")
        check(*problem(*shape, dtype, codes, see, extra=131072 // shape[5]), 131072, 4)


# many rows: wide tiles whose windows leave most of the context out
@pytest.mark.parametrize("shape,window,sinks", [
    (([3200], 2100, 16, 4, 128, 64, 64), 700, 4), (([2500], 2100, 16, 4, 64, 16, 16), 333, 70),
    (([1700, 1900], 1100, 8, 2, 128, 32, 16), 900, 17), (([2100], 2100, 8, 8, 64, 64, 32), 100, 1)],
    ids=lambda s: str(s))
@pytest.mark.parametrize("see", ["causal", "mixed"])
def test_wide_tiles(shape, window, sinks, see):
    say(f"case: wide window {shape} {window} {sinks} {see}")
    check(*problem(*shape, BF16, "e4m3", see), window, sinks)


@pytest.mark.parametrize("shape,window,sinks", [(([700, 900], 1, 32, 8, 128, 16, 16), 100, 4),
                                                (([700, 900], 4, 8, 2, 64, 16, 16), 33, 17),
                                                (([2600], 2100, 16, 4, 128, 16, 16), 300, 20)],
                         ids=lambda s: str(s))
@pytest.mark.parametrize("codes", ["e4m3", "int8"])
def test_pages_between_may_be_in_other_use(shape, window, sinks, codes):
    say(f"case: freed pages {shape} {codes}")
    lens, R, P = shape[0], shape[1], shape[5]
    pool, table, q, starts, ends = problem(*shape, BF16, codes)
    seen = serve_ref.window_seen(starts, ends, window, sinks, table.shape[1] * P)
    freed = table.clone()
    spoilt = set(range(pool.codes.shape[0]))
    for i in range(len(lens)):
        used = seen[i * R:(i + 1) * R].any(0).view(-1, P).any(1)
        spoilt -= set(table[i][used].tolist())
        # none, past the pool, and pages that hold nothing but NaN
        junk = torch.tensor([-1, 1 << 30, -(1 << 31), sorted(spoilt)[0]], dtype=torch.int32)
        freed[i] = torch.where(used, table[i], junk[torch.arange(table.shape[1]) % 4])
    spoilt = torch.tensor(sorted(spoilt))
    pool.codes[spoilt] = 0x7F
    pool.scales[spoilt] = math.nan
    # (a page that the table names twice is read, and masked)
    out, _ = check(pool, freed, q, starts, ends, window, sinks, want_table=table)
    assert bool(torch.isfinite(out.float()).all())


def test_a_window_past_the_range_is_the_range():
    # the same sums; keys may be cut into other parts, so that either call is within the
    # tolerance of the exact values, and the two within twice that
    pool, table, q, starts, ends = problem([700, 3, 129], 1, 32, 8, 128, 64, 32, BF16, "e4m3")
    args = (layout(pool), q.cuda(), pool.bytes().cuda(), table.cuda(), starts.cuda(), ends.cuda())
    cap = table.shape[1] * 64
    want, _, tol, _ = serve_ref.attend(pool, q, table, serve_ref.window_seen(starts, ends, cap, 0, cap))
    window, paged = mqa.mqa_attend_window(*args, 1 << 20), mqa.mqa_attend_paged(*args)
    assert ref.differs(window, want, tol) == 0 and ref.differs(paged, want, tol) == 0
    assert ref.differs(window, paged.double().cpu(), 2 * tol) == 0


@pytest.mark.parametrize("shape", [([20000, 9000], 1, 16, 2, 128, 64, 64), ([30000], 2, 8, 1, 64, 64, 64)],
                         ids=lambda s: "x".join(map(str, s[1:])))
def test_split_windows(shape):
    # few columns, long windows: keys in parts, sinks in the first
    say(f"case: split windows {shape}")
    pool, table, q, starts, ends = problem(*shape, BF16, "e4m3")
    for window, sinks in ((8000, 4), (12345, 300)):
        check(pool, table, q, starts, ends, window, sinks)
    Hq, (Hkv, D, P, B) = q.shape[1], pool.dims
    assert A._load().workspace_size_attend_call(len(shape[0]), shape[1], Hq, Hkv, D,
                                                8000 + 4 + shape[1] - 1, 0, 0) > 256


def test_out_lse_workspace_and_strides():
    pool, table, q, starts, ends = problem([900, 300], 2, 8, 2, 128, 64, 64, FP16, "e4m3")
    L, cache = layout(pool), pool.bytes(gap=256).cuda()[:, :ref.page_bytes(*pool.dims)]
    wide = torch.zeros(q.shape[0], q.shape[1] + 3, q.shape[2], dtype=q.dtype, device="cuda")
    wide[:, 1:-2] = q.cuda()
    out, lse = torch.empty_like(q, device="cuda"), torch.empty(q.shape[:2], device="cuda")
    n = mqa.workspace_size_attend(2, 2, 8, L, table.shape[1] * 64)
    work = torch.empty(n, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    args = (table.cuda(), starts.cuda(), ends.cuda(), 130, 5)
    torch.cuda.synchronize()
    got = mqa.mqa_attend_window(L, wide[:, 1:-2], cache, *args, out=out, lse=lse, workspace=work,
                                stream=stream)
    stream.synchronize()
    assert got.data_ptr() == out.data_ptr()
    want, wlse, tol, tol_lse = serve_ref.attend(
        pool, q, table, serve_ref.window_seen(starts, ends, 130, 5, table.shape[1] * 64))
    assert ref.differs(out, want, tol) == 0 and ref.differs(lse, wlse, tol_lse) == 0


def test_refusals():
    pool, table, q, starts, ends = problem([90], 2, 8, 2, 64, 16, 16, BF16, "e4m3")
    args = [layout(pool), q.cuda(), pool.bytes().cuda(), table.cuda(), starts.cuda(), ends.cuda()]
    for window, sinks in ((-1, 0), (8, -1), (1 << 31, 0), (8, 1 << 31)):
        with pytest.raises(ValueError):
            mqa.mqa_attend_window(*args, window, sinks)
    with pytest.raises(mqa.MQAError):
        mqa.mqa_attend_window(*args, 0)
    with pytest.raises(TypeError):
        mqa.mqa_attend_window(args[0], args[1].float(), *args[2:], 8)
