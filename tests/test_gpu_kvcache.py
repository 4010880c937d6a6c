"""Storing tokens into the paged 8-bit cache and reading them back, against
the 64-bit reference: codes and scales have to be equal."""
import math

import pytest
import torch

import attend_ref as ref
import fp8_mqa_logits_amd as mqa
from gpu_helpers import say

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def tokens(rows, Hkv, D, dtype, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(2, rows, Hkv, D, generator=g)
    x *= torch.exp2(torch.randn(2, rows, Hkv, 1, generator=g) * spread)
    return x[0].to(dtype), x[1].to(dtype)


def layout(pool):
    Hkv, D, P, B = pool.dims
    return mqa.KVLayout(Hkv, D, P, B, pool.kind)


def store(pool, k, v, table, starts, counts=None):
    """Both sides store; the whole pool's bytes have to be the same."""
    cache = pool.bytes().cuda()
    got = mqa.mqa_kv_append(layout(pool), k.cuda(), v.cuda(), cache, table.cuda(), starts.cuda(),
                            None if counts is None else counts.cuda())
    assert got is cache
    ref.append(pool, k, v, table, starts, counts)
    assert torch.equal(cache.cpu(), pool.bytes())
    return cache


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("starts,R,Hkv,D,P,B", [
    ([0], 1, 1, 64, 16, 16), ([7, 15, 16, 31], 1, 2, 128, 16, 16), ([0, 33], 64, 2, 64, 32, 32),
    ([5, 64, 127], 70, 3, 128, 64, 64), ([100], 200, 1, 128, 128, 32), ([3, 9], 2, 2, 64, 256, 128),
    ([5], 300, 1, 128, 512, 256)])
def test_append(starts, R, Hkv, D, P, B, dtype, codes):
    say(f"case: append {starts} {R} {Hkv} {D} {P} {B} {dtype} {codes}")
    table, pages = ref.make_table([s + R for s in starts], P, 2)
    pool = ref.Pool(pages, Hkv, D, P, B, codes, 3)
    pool.scales.log2_().round_().exp2_()  # scales as the operator writes them
    k, v = tokens(len(starts) * R, Hkv, D, dtype, 4)
    store(pool, k, v, table, torch.tensor(starts, dtype=torch.int32))


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
def test_token_by_token(codes):
    # a block filled one token at a time, louder and louder: its scale grows
    # and the tokens kept are rounded again
    say(f"case: token by token {codes}")
    table, pages = ref.make_table([40], 32, 2)
    pool = ref.Pool(pages, 2, 64, 32, 16, codes, 3)
    for t in range(40):
        k, v = tokens(1, 2, 64, BF16, 100 + t, 0.3)
        k, v = (k.float() * 2 ** (t / 4)).to(BF16), (v.float() * 2 ** (-t / 3)).to(BF16)
        store(pool, k, v, table, torch.tensor([t], dtype=torch.int32))


def test_counts_capacity_and_missing_pages():
    say("case: counts")
    table, pages = ref.make_table([60, 60, 60, 60, 60], 16, 2, extra=0)
    table[1, 2] = -1           # a page that is not there
    table[2, 1] = pages + 5    # nor this one
    pool = ref.Pool(pages, 2, 64, 16, 16, "e4m3", 3)
    pool.scales.log2_().round_().exp2_()
    k, v = tokens(5 * 48, 2, 64, BF16, 4)
    starts = torch.tensor([10, 20, 5, 50, -20], dtype=torch.int32)  # 50 + 48: past the table
    counts = torch.tensor([0, 48, 30, 99, 48], dtype=torch.int32)
    store(pool, k, v, table, starts, counts)
    counts[:] = -1
    store(pool, k, v, table, starts, counts)


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
def test_values_at_the_edges(codes):
    say(f"case: edges {codes}")
    top = 448.0 if codes == "e4m3" else 127.0
    table, pages = ref.make_table([16 * 12], 16, 2)
    pool = ref.Pool(pages, 1, 64, 16, 16, codes, 3)
    x = torch.zeros(16 * 12, 1, 64)
    x[0] = 0.0
    x[16, 0, :3] = torch.tensor([top, -top, 1.0])                       # the top exactly
    x[32, 0, :2] = torch.tensor([math.nextafter(top, 1e9), 1.0])        # just over it
    x[32] = torch.where(x[32] > top, torch.tensor(top * (1 + 2.0 ** -23)), x[32])
    x[48, 0, :3] = torch.tensor([math.inf, -math.inf, 3.0])
    x[64, 0, :2] = torch.tensor([math.nan, 3.0])
    x[80, 0, :] = math.nan
    x[96, 0, :2] = torch.tensor([3.0e38, -1.0])
    x[112, 0, :3] = torch.tensor([1e-38, 1e-40, -1e-45])
    x[128, 0, :] = torch.linspace(-top, top, 64)
    x[144, 0, :] = torch.arange(64) / 64 - 0.5                           # ties
    x[144, 0, 0] = top
    x[160, 0, 0] = math.inf
    for t in range(16):
        x[176 + t] = 0.5 * 2.0 ** -t
    store(pool, x, -x, table, torch.tensor([0], dtype=torch.int32))


def test_strided_tokens_and_interleaved_layers():
    say("case: strided append")
    table, pages = ref.make_table([100, 50], 32, 2)
    pool = ref.Pool(pages, 2, 64, 32, 32, "e4m3", 3)
    k, v = tokens(2 * 20, 2, 64, BF16, 4)
    qkv = torch.zeros(40, 8, 64, dtype=BF16, device="cuda")
    qkv[:, 4:6], qkv[:, 6:8] = k.cuda(), v.cuda()
    layers = torch.full((pages, 2, pool.bytes().shape[1]), 0x33, dtype=torch.uint8, device="cuda")
    layers[:, 1] = pool.bytes().cuda()
    starts = torch.tensor([80, 30], dtype=torch.int32)
    pool.scales.log2_().round_().exp2_()
    layers[:, 1] = pool.bytes().cuda()
    mqa.mqa_kv_append(layout(pool), qkv[:, 4:6], qkv[:, 6:8], layers[:, 1], table.cuda(), starts.cuda())
    ref.append(pool, k, v, table, starts)
    assert torch.equal(layers[:, 1].cpu(), pool.bytes())
    assert bool((layers[:, 0] == 0x33).all())


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("lens,R,Hkv,D,P,B", [
    ([1], 1, 1, 64, 16, 16), ([100, 40, 7], 45, 2, 128, 32, 16), ([300], 300, 3, 64, 64, 64)])
def test_read(lens, R, Hkv, D, P, B, dtype, codes):
    say(f"case: read {lens} {R} {Hkv} {D} {P} {B} {dtype} {codes}")
    table, pages = ref.make_table(lens, P, 2)
    pool = ref.Pool(pages, Hkv, D, P, B, codes, 3)
    starts = torch.tensor([n // 3 for n in lens], dtype=torch.int32)
    counts = torch.tensor([min(R, n - n // 3) for n in lens], dtype=torch.int32)
    got = mqa.mqa_kv_read(layout(pool), pool.bytes().cuda(), table.cuda(), starts.cuda(),
                          counts.cuda(), R, dtype=dtype)
    for w in (0, 1):
        want = torch.zeros(len(lens), R, Hkv, D, dtype=torch.float64)
        for i in range(len(lens)):
            pos = starts[i].long() + torch.arange(int(counts[i]))
            want[i, :len(pos)] = pool.tokens(table[i], pos)[w]
        # a code times its fp32 scale in fp32, then the type: at most two roundings
        want = want.view(-1, Hkv, D)
        tol = want.abs() * (2.0 ** -24 + {BF16: 2.0 ** -8, FP16: 2.0 ** -11, FP32: 0.0}[dtype]) + \
            (2.0 ** -25 if dtype == FP16 else 0)
        assert got[w].dtype == dtype and ref.differs(got[w], want, tol) == 0


def test_read_outside():
    say("case: read outside")
    table, pages = ref.make_table([64, 64], 16, 2, extra=0)
    table[1, 0] = -1
    pool = ref.Pool(pages, 1, 64, 16, 16, "e4m3", 3, nan_codes=True)
    starts = torch.tensor([-8, 8], dtype=torch.int32)
    k, v = mqa.mqa_kv_read(layout(pool), pool.bytes().cuda(), table.cuda(), starts.cuda(), None, 80,
                           dtype=FP32)
    k = k.view(2, 80, 64).cpu()
    assert bool((k[0, :8] == 0).all()) and bool((k[0, 72:] == 0).all())
    assert bool((k[1, :8] == 0).all()) and bool((k[1, 56:] == 0).all())
    want = pool.tokens(table[0], torch.arange(64))[0][:, 0]
    assert ref.differs(k[0, 8:72], want, want.abs() * 2.0 ** -24) == 0


def test_append_then_read_then_attend():
    # the cache as a user fills and uses it, a request growing to 150 tokens
    say("case: append, read, attend")
    table, pages = ref.make_table([150], 32, 2)
    pool = ref.Pool(pages, 2, 64, 32, 32, "e4m3", 3)
    L, cache = layout(pool), pool.bytes().cuda()
    k, v = tokens(150, 2, 64, BF16, 9, 0.3)
    at = 0
    for n in (100, 1, 1, 1, 40, 7):
        mqa.mqa_kv_append(L, k[at:at + n].cuda(), v[at:at + n].cuda(), cache, table.cuda(),
                          torch.tensor([at], dtype=torch.int32, device="cuda"))
        ref.append(pool, k[at:at + n], v[at:at + n], table, torch.tensor([at]))
        at += n
    rk, rv = mqa.mqa_kv_read(L, cache, table.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda"),
                             None, 150)
    # codes are within half a step of 2^-3 of the block's loudest binade or 2^-4
    # relative: far nearer than this
    assert float((rk.cpu().double() - k.double()).norm() / k.double().norm()) < 0.06
    q = tokens(3, 4, 64, BF16, 11, 0.0)[0]
    starts, ends = torch.zeros(3, dtype=torch.int32), torch.tensor([148, 149, 150], dtype=torch.int32)
    out = mqa.mqa_attend_paged(L, q.cuda(), cache, table.cuda(), starts.cuda(), ends.cuda())
    want, _, tol, _ = ref.attend(pool, q, table, starts, ends)
    assert ref.differs(out, want, tol) == 0


def test_binding_refusals():
    pool = ref.Pool(4, 2, 64, 16, 16, "e4m3", 3)
    L, cache = layout(pool), pool.bytes().cuda()
    table = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    k = torch.zeros(4, 2, 64, dtype=BF16, device="cuda")
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        mqa.mqa_kv_append(L, k.int(), k.int(), cache, table, z)
    with pytest.raises(TypeError):
        mqa.mqa_kv_append(L, k, k.half(), cache, table, z)
    with pytest.raises(ValueError):
        mqa.mqa_kv_append(L, k[:, :1], k[:, :1], cache, table, z)
    with pytest.raises(ValueError):
        mqa.mqa_kv_append(L, k, k, cache, table, z[:0])
    with pytest.raises(ValueError):
        mqa.mqa_kv_append(L, k, k[:3], cache, table, z)
    with pytest.raises(TypeError):
        mqa.mqa_kv_read(L, cache, table, z, None, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        mqa.mqa_kv_read(L, cache, table, z, None, 0)
    with pytest.raises(ValueError):
        mqa.KVLayout(2, 96).page_bytes
    with pytest.raises(ValueError):
        mqa.KVLayout(2, 64, codes="fp4")
    with pytest.raises(mqa.MQAError) as e:
        mqa.mqa_kv_append(L, k[:0], k[:0], cache, table, z)
    assert e.value.code in (1, 3)  # no rows: also no memory


@pytest.mark.parametrize("R,Hq", [(1, 8), (3, 32), (40, 16)])
@pytest.mark.parametrize("codes", ["e4m3", "int8"])
def test_a_captured_step_stores_and_then_reads_what_it_stored(R, Hq, codes):
    # append, attention over the range and over a list, and read back in one graph,
    # replayed as the requests grow; every replay against the eager calls
    say(f"case: captured step {R} {Hq} {codes}")
    L = mqa.KVLayout(2, 128, 32, 16, codes)
    table, pages = ref.make_table([400, 300], 32, 2)
    table = table.cuda()
    caches = [torch.zeros(pages, L.page_bytes, dtype=torch.uint8, device="cuda") for _ in range(2)]
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.zeros(2 * R, 2, 128, dtype=BF16, device="cuda") for _ in range(2))
    q = torch.zeros(2 * R, Hq, 128, dtype=BF16, device="cuda")
    first = torch.zeros(2, dtype=torch.int32, device="cuda")
    starts = torch.zeros(2 * R, dtype=torch.int32, device="cuda")
    ends = torch.zeros_like(starts)
    idx = torch.arange(64, dtype=torch.int32, device="cuda").repeat(2 * R, 1)

    def step(cache):
        mqa.mqa_kv_append(L, k, v, cache, table, first)
        out = [mqa.mqa_attend_paged(L, q, cache, table, starts, ends),
               mqa.mqa_attend_topk(L, q, cache, table, idx, starts, ends)]
        return out + list(mqa.mqa_kv_read(L, cache, table, first, None, R))

    step(caches[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(caches[0])
    for i in range(6):
        first.copy_(torch.tensor([i * R, 37 + i * R], dtype=torch.int32))
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda") * 2.0 ** (i % 3))
        ends.copy_((first[:, None] + 1 + torch.arange(R, device="cuda")).flatten())
        starts.copy_((ends - 70).clamp(min=0))
        for o in got:
            o.zero_()
        graph.replay()
        want = step(caches[1])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)), i
        if i == 0:  # (the call before the capture stored zeros into the first one)
            caches[0].copy_(caches[1])
        assert torch.equal(*caches)
