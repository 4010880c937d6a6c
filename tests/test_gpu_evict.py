"""Eviction from the paged 8-bit cache: weights that positions receive against the
formula in 64 bits, selection against a sort, moving against reading and storing
again."""
import math

import pytest
import torch

import attend_ref as ref
import fp8_mqa_logits_amd as mqa
import serve_ref
from gpu_helpers import say
from test_gpu_attend import SHAPES, layout, problem

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


# ---------------------------------------------------------------- weighing

def weigh_ref(pool, q, table, starts, ends, lse, scale=None):
    """(weights [N, cap], tolerance) in float64. A term's exponent is off by the fp32 dot
    product, D 2^-24 of sum_d |q_d k_d|, and by roundings of its products and differences
    (to base 2, six of half a last place of at most |S| + |lse| + 1 together); sums are
    of positive fp32 terms, one rounding each."""
    Hkv, D, P, B = pool.dims
    rows, Hq, _ = q.shape
    N, cap = table.shape[0], table.shape[1] * P
    R, G = rows // N, Hq // Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    s, e = serve_ref.ranges(starts, ends, min(cap, 1 << 20))
    W, tol = torch.zeros(N, cap, dtype=torch.float64), torch.zeros(N, cap, dtype=torch.float64)
    for i in range(N):
        r = slice(i * R, (i + 1) * R)
        at = torch.arange(cap)
        seen = (at >= s[r]) & (at < e[r])
        used = seen.any(0).nonzero()[:, 0]
        if not len(used):
            continue
        k = pool.tokens(table[i], used)[0].transpose(0, 1)  # [Hkv, n, D]
        x = q[r].double().view(R, Hkv, G, D).transpose(0, 1).reshape(Hkv, -1, D)
        S = x @ k.transpose(1, 2) * scale
        L = lse[r].double().view(R, Hkv, G).transpose(0, 1).reshape(Hkv, -1, 1)
        ok = seen[:, None, used].expand(-1, G, -1).reshape(1, -1, len(used)) & (L > -math.inf)
        t = torch.where(ok, torch.exp(S - torch.where(ok, L, 0.0)), 0.0)
        off = D * 2.0 ** -24 * scale * (x.abs() @ k.abs().transpose(1, 2)) + \
            6 * 2.0 ** -24 * (S.abs() + L.abs() + 1)
        W[i, used] = t.sum((0, 1))
        tol[i, used] = torch.where(ok, t * torch.expm1(off), 0.0).sum((0, 1)) + \
            2.0 ** -24 * R * Hq * W[i, used]
    return W, tol


def check_weigh(pool, table, q, starts, ends, lse=None, scale=None, width=None, seed=5, **kw):
    N, cap = table.shape[0], table.shape[1] * pool.dims[2]
    if lse is None:
        lse = mqa.mqa_attend_paged(layout(pool), q.cuda(), pool.bytes().cuda(), table.cuda(),
                                   starts.cuda(), ends.cuda(), scale=scale, return_lse=True)[1].cpu()
    want, tol = weigh_ref(pool, q, table, starts, ends, lse, scale)
    width = cap if width is None else width
    before = torch.rand(N, width, generator=torch.Generator().manual_seed(seed))
    w = before.cuda()
    got = mqa.mqa_kv_weigh(layout(pool), q.cuda(), pool.bytes().cuda(), table.cuda(), starts.cuda(),
                           ends.cuda(), lse.cuda(), w, scale=scale, **kw)
    torch.cuda.synchronize()
    assert got.data_ptr() == w.data_ptr()
    some = min(width, cap)
    total = before.double()
    total[:, :some] += want[:, :some]
    bound = 2.0 ** -24 * total
    bound[:, :some] += tol[:, :some]
    assert ref.differs(w, total, bound) == 0
    # what no row sees keeps its bits
    assert torch.equal(w.cpu()[:, :some][want[:, :some] == 0], before[:, :some][want[:, :some] == 0])
    assert torch.equal(w.cpu()[:, some:], before[:, some:])
    return w


@pytest.mark.parametrize("dtype,codes", [(BF16, "e4m3"), (FP16, "int8"), (FP16, "e4m3"), (BF16, "int8")])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[1:])))
def test_weights_of_ranges(shape, dtype, codes):
    for see in ("causal", "window") if shape[1] > 1 else ("causal",):
        say(f"case: weigh {shape} {dtype} {codes} {see}")
        check_weigh(*problem(*shape, dtype, codes, see))


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[1] in (4, 7, 40, 130)],
                         ids=lambda s: "x".join(map(str, s[1:])))
@pytest.mark.parametrize("see", ["mixed", "full"])
def test_weights_of_any_range(shape, see):
    say(f"case: weigh {shape} {see}")
    check_weigh(*problem(*shape, BF16, "e4m3", see))


@pytest.mark.parametrize("shape", [([2000], 700, 8, 2, 128, 64, 64), ([900, 1500], 600, 12, 12, 64, 16, 16),
                                   ([3100], 333, 28, 4, 128, 32, 16), ([700], 700, 5, 1, 64, 128, 64)],
                         ids=lambda s: "x".join(map(str, s[1:])))
@pytest.mark.parametrize("see", ["causal", "window", "mixed"])
def test_weights_of_chunks(shape, see):
    say(f"case: weigh chunk {shape} {see}")
    check_weigh(*problem(*shape, FP16, "e4m3", see))


def test_a_row_s_heads_share_out_their_number():
    pool, table, q, starts, ends = problem([777, 41], 3, 32, 8, 128, 64, 64, BF16, "e4m3")
    args = (layout(pool), q.cuda(), pool.bytes().cuda(), table.cuda(), starts.cuda(), ends.cuda())
    lse = mqa.mqa_attend_paged(*args, return_lse=True)[1]
    w = mqa.mqa_kv_weigh(*args, lse, torch.zeros(2, table.shape[1] * 64, device="cuda"))
    # a term is off by 2^-18 (lse's tolerance) and as much again here
    assert float((w.double().sum(1) - 3 * 32).abs().max()) < 3 * 32 * (2.0 ** -17 + 2.0 ** -14)


@pytest.mark.parametrize("rows", [4, 200])
def test_rows_without_weight_nan_and_unseen_keys(rows):
    pool, table, q, starts, ends = problem([500], rows, 8, 2, 128, 64, 16, BF16, "e4m3", "window")
    lse = mqa.mqa_attend_paged(layout(pool), q.cuda(), pool.bytes().cuda(), table.cuda(), starts.cuda(),
                               ends.cuda(), return_lse=True)[1].cpu()
    lse[1, 3], lse[2] = -math.inf, -math.inf
    # NaN keys where no row sees them: in the first and the last blocks in reach, and past the end
    lo, hi = int(starts.min()), int(ends.max())
    assert lo >= 1
    for at in {lo - 1, hi}:
        if at < table.shape[1] * 64 and int(table[0, at // 64]) >= 0:
            pool.codes[int(table[0, at // 64]), 0, :, at % 64] = 0x7F
    say(f"case: weigh with dead rows {rows}")
    check_weigh(pool, table, q, starts, ends, lse)
    # one that a single row sees: only that position becomes NaN
    at = lo
    pool.codes[int(table[0, at // 64]), 0, 0, at % 64, 7] = 0x7F
    w = torch.zeros(1, table.shape[1] * 64, device="cuda")
    mqa.mqa_kv_weigh(layout(pool), q.cuda(), pool.bytes().cuda(), table.cuda(), starts.cuda(), ends.cuda(),
                     lse.cuda(), w)
    assert torch.isnan(w[0]).nonzero()[:, 0].tolist() == [at]


def test_weights_narrower_and_wider_than_the_table():
    shape = ([300, 41], 4, 10, 2, 64, 32, 32)
    for width in (1, 17, 100, 1000):
        check_weigh(*problem(*shape, BF16, "e4m3"), width=width)


def test_weighing_gives_the_same_bits_and_replays():
    for R in (2, 300):
        pool, table, q, starts, ends = problem([900, 700], R, 8, 2, 128, 64, 64, BF16, "e4m3")
        L = layout(pool)
        args = (L, q.cuda(), pool.bytes().cuda(), table.cuda(), starts.cuda(), ends.cuda())
        lse = mqa.mqa_attend_paged(*args, return_lse=True)[1]
        w = torch.zeros(2, table.shape[1] * 64, device="cuda")
        want = mqa.mqa_kv_weigh(*args, lse, w.clone())
        work = torch.empty(mqa.workspace_size_weigh(2, R, 8, L, table.shape[1] * 64), dtype=torch.uint8,
                           device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = w.clone()
        torch.cuda.synchronize()
        mqa.mqa_kv_weigh(*args, lse, got, workspace=work, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mqa.mqa_kv_weigh(*args, lse, w, workspace=work)
        for k in range(3):
            w.zero_()
            graph.replay()
            assert torch.equal(w, want)


# --------------------------------------------------------------- selection

def select_ref(w, lengths, keep, sinks, recent):
    lists, kept = [], torch.zeros_like(w)
    for i, n in enumerate(lengths.tolist()):
        n = min(max(n, 0), w.shape[1])
        must = [j for j in range(n) if j < sinks or j >= n - recent]
        chosen = set(must)
        rest = [j for j in range(n) if j not in chosen]
        value = w[i].tolist()
        rest.sort(key=lambda j: (-math.inf if math.isnan(value[j]) else 0,
                                 0 if math.isnan(value[j]) else -value[j], j))
        chosen = sorted(must + rest[:max(0, min(n, keep) - len(must))])
        lists.append(chosen)
        kept[i, :len(chosen)] = w[i, chosen]
    return lists, kept


def check_select(w, lengths, keep, sinks, recent):
    lists, want = select_ref(w, lengths, keep, sinks, recent)
    d = w.cuda()
    kept = torch.full_like(d, 7.0)
    positions, counts = mqa.mqa_kv_select(d, lengths.cuda(), keep, sinks, recent, kept=kept)
    alone = mqa.mqa_kv_select(d, lengths.cuda(), keep, sinks, recent)
    torch.cuda.synchronize()
    assert counts.tolist() == [len(x) for x in lists]
    for i, x in enumerate(lists):
        assert positions[i].tolist() == x + [-1] * (keep - len(x)), i
    assert torch.equal(kept.cpu().view(torch.int32), want.view(torch.int32))
    assert torch.equal(alone[0], positions) and torch.equal(alone[1], counts)
    assert torch.equal(d.cpu().view(torch.int32), w.view(torch.int32))


@pytest.mark.parametrize("width", [1, 63, 64, 65, 1000, 1024, 1025, 5000, 70000])
def test_selection(width):
    g = torch.Generator().manual_seed(width)
    w = torch.exp(torch.randn(6, width, generator=g) * 2 - 6)
    lengths = torch.tensor([width, 0, 1, width // 2, width + 100, -5]).int()
    for keep, sinks, recent in ((1, 0, 0), (5, 4, 1), (64, 4, 16), (width // 3 + 3, 2, 1),
                                (width + 7, 0, 0), (max(2, width - 1), 1, 0)):
        say(f"case: select {width} {keep} {sinks} {recent}")
        check_select(w, lengths, keep, sinks, recent)


@pytest.mark.parametrize("width", [777, 3000])
def test_selection_with_equal_weights(width):
    g = torch.Generator().manual_seed(1)
    few = torch.randint(0, 4, (5, width), generator=g).float() * 0.25
    few[1] = 0.0  # all equal
    few[2, ::2] = -0.0
    few[3] = few[3].neg()
    lengths = torch.tensor([width, width, width, width, width - 5]).int()
    for keep, sinks, recent in ((10, 0, 0), (width // 2, 4, 9), (300, 0, 300), (300, 300, 0), (300, 150, 150)):
        check_select(few, lengths, keep, sinks, recent)


def test_selection_of_any_number():
    g = torch.Generator().manual_seed(2)
    w = torch.randint(-(1 << 31), (1 << 31) - 1, (4, 2000), generator=g).int().view(torch.float32)
    w[0, 5:40:5] = math.inf
    w[1, 3::50] = -math.inf
    w[2, 100:1500] = math.nan
    w[3] = torch.randn(2000, generator=g) * 1e-42  # subnormals
    lengths = torch.full((4,), 2000).int()
    for keep in (3, 100, 1999):
        check_select(w, lengths, keep, 2, 1)


def test_selection_into_a_graph():
    g = torch.Generator().manual_seed(3)
    w = torch.rand(3, 900, generator=g).cuda()
    lengths = torch.tensor([900, 20, 500]).int().cuda()
    kept = torch.empty_like(w)
    mqa.mqa_kv_select(w, lengths, 100, 4, 10, kept=kept)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        positions, counts = mqa.mqa_kv_select(w, lengths, 100, 4, 10, kept=kept)
    for k in range(3):
        w.copy_(torch.rand(3, 900, generator=g))
        graph.replay()
        got = positions.clone(), counts.clone(), kept.clone()
        other = torch.empty_like(kept)
        want = mqa.mqa_kv_select(w, lengths, 100, 4, 10, kept=other)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], other)


# ------------------------------------------------------------------ moving

def lists_of(lens, starts, share, seed, width=None):
    g = torch.Generator().manual_seed(seed)
    lists = []
    for n, s in zip(lens, starts):
        some = (torch.rand(max(n - s, 0), generator=g) < share).nonzero()[:, 0] + s
        lists.append(some)
    width = max(1, max(len(x) for x in lists)) if width is None else width
    out = torch.full((len(lens), width), -1, dtype=torch.int32)
    for i, x in enumerate(lists):
        out[i, :min(len(x), width)] = x[:width].int()
    return out, torch.tensor([min(len(x), width) for x in lists]).int()


def stored_again(L, cache, table, listed, counts, starts):
    """What reading and storing give: the cache's bytes, by the package's own calls."""
    N, width = listed.shape
    cap = table.shape[1] * L.page_size
    zero = torch.zeros(N, dtype=torch.int32, device="cuda")
    k, v = mqa.mqa_kv_read(L, cache, table, zero, None, cap, dtype=torch.float32)
    at = listed.long()
    ok = (at >= 0) & (at < cap)
    row = torch.arange(N, device="cuda")[:, None] * cap + at.clamp(0, cap - 1)

    def pick(t):
        return torch.where(ok.view(-1, 1, 1), t[row.view(-1)], 0.0)

    return mqa.mqa_kv_append(L, pick(k), pick(v), cache.clone(), table,
                             zero if starts is None else starts, counts)


def check_keep(pool, table, listed, counts, starts=None, workspace=None):
    L = layout(pool)
    P, B = pool.dims[2:]
    cache, table = pool.bytes().cuda(), table.cuda()
    d = [listed.cuda(), counts.cuda(), None if starts is None else starts.cuda()]
    want = stored_again(L, cache, table, *d)
    # blocks whose tokens all stay where they are keep their bytes
    as_it_was = cache.clone()
    n = 2 * pool.dims[0] * P * pool.dims[1]
    codes = (slice(None), slice(0, n))
    want_codes, was_codes = want[codes].view(-1, 2, pool.dims[0], P, pool.dims[1]), \
        as_it_was[codes].view(-1, 2, pool.dims[0], P, pool.dims[1])
    m = n + 2 * pool.dims[0] * (P // B) * 4
    want_scales, was_scales = (t[:, n:m].view(torch.float32).view(-1, 2, pool.dims[0], P // B)
                               for t in (want, as_it_was))
    for i in range(len(listed)):
        s = 0 if starts is None else int(starts[i])
        c = min(max(int(counts[i]), 0), listed.shape[1])
        for b in range(max(s, 0) // B, (s + c - 1) // B + 1):
            lo, hi = max(b * B, s), min(b * B + B, s + c)
            if lo >= hi or b * B >= table.shape[1] * P:
                continue
            if listed[i, lo - s:hi - s].tolist() == list(range(lo, hi)):
                page, slot = int(table[i, b * B // P]), b * B % P
                if 0 <= page < len(cache):
                    want_codes[page, :, :, slot:slot + B] = was_codes[page, :, :, slot:slot + B]
                    want_scales[page, :, :, slot // B] = was_scales[page, :, :, slot // B]
    want[codes] = want_codes.reshape(len(want), -1)
    want[:, n:m] = want_scales.contiguous().view(torch.uint8).view(len(want), -1)
    got = mqa.mqa_kv_keep(L, cache, table, *d, workspace=workspace)
    torch.cuda.synchronize()
    assert got.data_ptr() == cache.data_ptr()
    assert torch.equal(cache, want)
    return cache


KEEP_SHAPES = [
    # lens, Hkv, D, P, B
    ([1], 1, 64, 16, 16), ([700, 3, 129, 128], 8, 128, 64, 32), ([333, 90], 12, 128, 128, 64),
    ([1500, 1400], 1, 128, 16, 16), ([600], 2, 64, 256, 256), ([9001], 4, 128, 64, 64),
    ([2000], 2, 128, 1024, 1024), ([40000], 2, 64, 64, 16)]


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("shape", KEEP_SHAPES, ids=lambda s: "x".join(map(str, s[1:])))
def test_moving(shape, codes):
    lens, Hkv, D, P, B = shape
    for share in (0.03, 0.5, 0.97, 1.0):
        say(f"case: keep {shape} {codes} {share}")
        table, pages = ref.make_table(lens, P, 1)
        pool = ref.Pool(pages, Hkv, D, P, B, codes, 1, nan_codes=share == 0.5)
        check_keep(pool, table, *lists_of(lens, [0] * len(lens), share, 3))


@pytest.mark.parametrize("codes", ["e4m3", "int8"])
@pytest.mark.parametrize("shape", [([40], 2, 64, 16, 16), ([700, 63, 129, 128], 8, 128, 64, 32),
                                   ([333, 90], 3, 128, 128, 64), ([1100, 900], 1, 64, 1024, 512)],
                         ids=lambda s: "x".join(map(str, s[1:])))
def test_moving_behind_what_stays(shape, codes):
    # accepted drafts: a few tokens behind a context that ends anywhere in a block
    lens, Hkv, D, P, B = shape
    for back, share in ((1, 1.0), (5, 0.6), (13, 0.4), (60, 0.3)):
        starts = [max(0, n - back) for n in lens]
        say(f"case: accept {shape} {codes} {back} {share}")
        table, pages = ref.make_table(lens, P, 2)
        pool = ref.Pool(pages, Hkv, D, P, B, codes, 2)
        listed, counts = lists_of(lens, starts, share, back, width=back)
        check_keep(pool, table, listed, counts, torch.tensor(starts).int())


def test_moving_by_the_definition_in_64_bits():
    # (the pool's scales are no powers of two: a value is rounded once in fp32, and so are
    # 1 / scale, where a block keeps its scale, and the quotient: together less than 2^-21
    # of it, so that a code is as near to the value as the nearest is, but for twice that)
    lens, Hkv, D, P, B = [130, 70], 2, 64, 32, 16
    for codes in ("e4m3", "int8"):
        table, pages = ref.make_table(lens, P, 4)
        pool = ref.Pool(pages, Hkv, D, P, B, codes, 4)
        starts = torch.tensor([3, 21]).int()
        listed, counts = lists_of(lens, starts.tolist(), 0.4, 5)
        cache = check_keep(pool, table, listed, counts, starts).cpu()
        before = [pool.tokens(table[i], torch.arange(lens[i])) for i in range(2)]
        k, v = (torch.stack([pool.tokens(table[i], listed[i].long().clamp(min=0))[w] for i in range(2)])
                .view(-1, Hkv, D) for w in (0, 1))
        ref.append(pool, k, v, table, starts, counts)  # the scales that should stand there
        n = 2 * Hkv * P * D
        got = ref.Pool(pages, Hkv, D, P, B, codes, 4)
        got.codes = cache[:, :n].view(got.codes.shape)
        got.scales = cache[:, n:n + 2 * Hkv * (P // B) * 4].contiguous().view(torch.float32).view(got.scales.shape)
        assert torch.equal(got.scales, pool.scales)
        for i in range(2):
            s, m = int(starts[i]), int(counts[i])
            at = torch.arange(s + m)
            source = torch.cat((at[:s], listed[i, :m].long()))
            page, slot = table[i].long()[at // P], at % P
            for w, x in enumerate(got.tokens(table[i], at)):
                scale = pool.scales[page, w, :, slot // B].double()[..., None]
                y = before[i][w][source]
                best = (ref.nearest(y / scale, codes) * scale - y).abs()
                assert bool(((x - y).abs() <= best + 2.0 ** -20 * y.abs()).all())


@pytest.mark.parametrize("many", [False, True])
def test_entries_without_a_position_and_pages_that_are_none(many):
    lens, Hkv, D, P, B = [500, 300], 2, 64, 16, 16
    table, pages = ref.make_table(lens, P, 6)
    pool = ref.Pool(pages, Hkv, D, P, B, "e4m3", 6)
    listed, counts = lists_of(lens, [0, 0], 0.5 if many else 0.05, 7)
    table[0, 20], table[1, 9] = -1, pages + 5  # sources without a page: zeros
    counts[1] += 3  # past the list: clamped
    listed[0, 2] = -1
    listed[0, int(counts[0]) - 1] = 1 << 20
    check_keep(pool, table, listed, counts)
    if many:  # places without a page are not written
        table[0, 3] = -1
        check_keep(pool, table, listed, counts)
    check_keep(pool, table, listed, torch.tensor([0, -4]).int())
    check_keep(pool, table, listed, counts, torch.tensor([-20, table.shape[1] * P - 4]).int())


def test_a_workspace_of_another_call_and_replays():
    lens, Hkv, D, P, B = [900, 300], 2, 128, 64, 64
    table, pages = ref.make_table(lens, P, 8)
    pool = ref.Pool(pages, Hkv, D, P, B, "int8", 8)
    L = layout(pool)
    work = torch.full((mqa.workspace_size_keep(8, 2000, L),), 0xFF, dtype=torch.uint8, device="cuda")
    for share in (0.9, 0.1):
        check_keep(pool, table, *lists_of(lens, [0, 0], share, 9), workspace=work)
    listed, counts = (t.cuda() for t in lists_of(lens, [0, 0], 0.4, 10))
    fresh, cache = pool.bytes().cuda(), pool.bytes().cuda()
    want = mqa.mqa_kv_keep(L, fresh.clone(), table.cuda(), listed, counts)
    d = table.cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mqa.mqa_kv_keep(L, cache, d, listed, counts, workspace=work)
    for k in range(3):
        cache.copy_(fresh)
        work.fill_(k)
        graph.replay()
        assert torch.equal(cache, want)
    side = torch.cuda.Stream()
    cache.copy_(fresh)
    torch.cuda.synchronize()
    mqa.mqa_kv_keep(L, cache, d, listed, counts, stream=side)
    side.synchronize()
    assert torch.equal(cache, want)


def test_refusals():
    pool, table, q, starts, ends = problem([90], 2, 8, 2, 64, 16, 16, BF16, "e4m3")
    L, cache, t = layout(pool), pool.bytes().cuda(), table.cuda()
    q, s, e = q.cuda(), starts.cuda(), ends.cuda()
    lse, w = torch.zeros(2, 8, device="cuda"), torch.zeros(1, 96, device="cuda")
    for bad in ((q.float(), cache, t, s, e, lse, w), (q, cache, t, s.long(), e, lse, w),
                (q, cache, t, s, e, lse.double(), w), (q, cache, t, s, e, lse, w.double())):
        with pytest.raises(TypeError):
            mqa.mqa_kv_weigh(L, *bad)
    for bad in ((q, cache, t, s, e, lse[:1], w), (q, cache, t, s, e, lse, w[0]), (q, cache, t, s, e, lse, w.cpu()),
                (q, cache, t, s, e, lse, torch.zeros(2, 96, device="cuda")),
                (q, cache, t, s, e, lse, torch.zeros(1, 192, device="cuda")[:, ::2])):
        with pytest.raises(ValueError):
            mqa.mqa_kv_weigh(L, *bad)
    n = torch.tensor([90]).int().cuda()
    for bad in ((w.double(), n, 8), (w, n.long(), 8)):
        with pytest.raises(TypeError):
            mqa.mqa_kv_select(*bad)
    for bad in ((w[0], n, 8), (w.cpu(), n, 8), (w, n[:0], 8), (w, n, -1), (w, n, 8, -1), (w, n, 8, 0, 1 << 31)):
        with pytest.raises(ValueError):
            mqa.mqa_kv_select(*bad)
    with pytest.raises(ValueError):
        mqa.mqa_kv_select(w, n, 8, kept=w)
    for bad in ((w, n, 0), (w, n, 8, 5, 4), (w, n, (1 << 20) + 1)):
        with pytest.raises(mqa.MQAError):
            mqa.mqa_kv_select(*bad)
    listed, c = torch.zeros(1, 8, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    for bad in ((listed.long(), c), (listed, c.long()), (listed, c, c.long())):
        with pytest.raises(TypeError):
            mqa.mqa_kv_keep(L, cache, t, *bad)
    for bad in ((listed[0], c), (listed.expand(2, -1), c), (listed, c.expand(2)), (listed.cpu(), c)):
        with pytest.raises(ValueError):
            mqa.mqa_kv_keep(L, cache, t, *bad)
    with pytest.raises(mqa.MQAError):
        mqa.mqa_kv_keep(L, cache, t, listed, c, workspace=torch.empty(128, dtype=torch.uint8, device="cuda"))
