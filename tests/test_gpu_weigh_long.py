"""Weighing few columns in tables with room for many positions, where every wave has keys of
its own, against the formula in 64 bits. Tolerances: test_gpu_evict.weigh_ref."""
import pytest
import torch

import fp8_mqa_logits_amd as mqa
from gpu_helpers import say
from test_gpu_attend import layout, problem
from test_gpu_evict import check_weigh

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16
BOTH = [(BF16, "e4m3"), (FP16, "int8"), (FP16, "e4m3"), (BF16, "int8")]


def roomy(shape, *a, **kw):
    """A problem whose tables have room for so many positions that four workgroups of 256
    keys a compute unit have work (the limit of the other form)."""
    lens, P = shape[0], shape[5]
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    out = problem(*shape, *a, extra=-(-4 * 256 * cus // (len(lens) * P)), **kw)
    assert len(lens) * out[1].shape[1] * P >= 4 * 256 * cus
    assert shape[1] * shape[2] // shape[3] <= 384
    return out


SHAPES = [
    # lens, R, Hq, Hkv, D, P, B
    ([1, 17, 63, 64, 65], 1, 8, 2, 128, 64, 64), ([700, 3, 255, 257, 1000], 1, 32, 8, 64, 64, 32),
    ([1300, 411], 3, 10, 2, 64, 32, 32), ([900, 777, 513], 3, 64, 1, 128, 16, 16),
    ([260, 1500], 40, 16, 2, 128, 64, 16), ([333, 90, 600, 40], 40, 12, 12, 64, 128, 128),
    ([999], 5, 5, 1, 128, 256, 64), ([2100, 2049, 1, 640], 1, 96, 3, 128, 64, 64)]


@pytest.mark.parametrize("dtype,codes", BOTH)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[1:])))
def test_weights(shape, dtype, codes):
    for see in ("causal", "window", "mixed", "full") if shape[1] > 1 else ("causal",):
        say(f"case: weigh long {shape} {dtype} {codes} {see}")
        check_weigh(*roomy(shape, dtype, codes, see))


@pytest.mark.parametrize("shape", SHAPES[1:4], ids=lambda s: "x".join(map(str, s[1:])))
@pytest.mark.parametrize("width", [1, 17, 300])
def test_narrow_weights(shape, width):
    check_weigh(*roomy(shape, BF16, "e4m3"), width=width)


def test_ranges_from_anywhere():
    # one row a request, from positions that are no multiple of 16, 64 or 256
    shape = ([1700, 1234, 900, 333], 1, 16, 2, 128, 64, 32)
    pool, table, q, starts, ends = roomy(shape, BF16, "e4m3")
    for first, last in (([5, 261, 899, 0], [1700, 1234, 900, 1]), ([63, 64, 65, 300], [600, 70, 321, 299])):
        check_weigh(pool, table, q, torch.tensor(first).int(), torch.tensor(last).int())


def test_nan_keys_beside_and_inside():
    shape = ([900, 500], 4, 8, 2, 128, 64, 16)
    pool, table, q, starts, ends = roomy(shape, BF16, "e4m3", "window")
    args = [layout(pool), q.cuda(), pool.bytes().cuda(), table.cuda(), starts.cuda(), ends.cuda()]
    lse = mqa.mqa_attend_paged(*args, return_lse=True)[1].cpu()
    lse[1, 3], lse[6] = -float("inf"), -float("inf")
    for i in (0, 1):
        lo, hi = int(starts[4 * i]), int(ends[4 * i + 3])
        for at in (lo - 1, hi):
            if at < shape[0][i]:
                pool.codes[int(table[i, at // 64]), 0, :, at % 64] = 0x7F
    say("case: weigh long beside NaN")
    check_weigh(pool, table, q, starts, ends, lse)
    at = int(starts[0])
    pool.codes[int(table[0, at // 64]), 0, 1, at % 64, 100] = 0x7F
    w = torch.zeros(2, table.shape[1] * 64, device="cuda")
    mqa.mqa_kv_weigh(args[0], args[1], pool.bytes().cuda(), *args[3:], lse.cuda(), w)
    assert torch.isnan(w).nonzero().tolist() == [[0, at]]


def test_the_same_bits_and_replays():
    shape = ([1900, 700], 2, 8, 2, 128, 64, 64)
    pool, table, q, starts, ends = roomy(shape, FP16, "int8")
    args = (layout(pool), q.cuda(), pool.bytes().cuda(), table.cuda(), starts.cuda(), ends.cuda())
    lse = mqa.mqa_attend_paged(*args, return_lse=True)[1]
    w = torch.zeros(2, table.shape[1] * 64, device="cuda")
    want = mqa.mqa_kv_weigh(*args, lse, w.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mqa.mqa_kv_weigh(*args, lse, w)
    for _ in range(3):
        w.zero_()
        graph.replay()
        assert torch.equal(w, want)
