"""The operators around attention together, as a serving step uses them: normed and
rotated keys stored, attended to, weighed, cut to the heaviest and attended to again;
trees verified and their accepted paths moved; captured and replayed."""
import math
import os
import sys

import pytest
import torch

import attend_ref as ref
import fp8_mqa_logits_amd as mqa
import serve_ref
from gpu_helpers import say
from test_gpu_evict import weigh_ref

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


def pool_of(cache, L):
    """What the cache's bytes stand for, as a reference pool."""
    pool = ref.Pool(len(cache), L.kv_heads, L.head_dim, L.page_size, L.block, L.codes, 0)
    n = pool.codes[0].numel()
    m = pool.scales[0].numel() * 4
    c = cache.cpu()
    pool.codes = c[:, :n].reshape(pool.codes.shape)
    pool.scales = c[:, n:n + m].contiguous().view(torch.float32).view(pool.scales.shape)
    return pool


def inputs(N, R, Hq, Hkv, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N * R, Hq + 2 * Hkv, D, generator=g).to(dtype).cuda()
    w = [(1 + 0.2 * torch.randn(D, generator=g)).to(dtype).cuda() for _ in range(2)]
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], w


@pytest.mark.parametrize("lens,Hq,Hkv,D,P,B,codes,dtype", [
    ([700, 433], 16, 4, 128, 64, 32, "e4m3", BF16), ([600], 12, 12, 64, 16, 16, "int8", FP16),
    ([1500, 900, 1201], 8, 2, 128, 32, 16, "e4m3", FP16)])
def test_store_weigh_cut_and_attend(lens, Hq, Hkv, D, P, B, codes, dtype):
    say(f"case: serving step {lens} {Hq} {Hkv} {D} {codes} {dtype}")
    N, R = len(lens), max(lens)
    L = mqa.KVLayout(Hkv, D, P, B, codes)
    table, pages = ref.make_table(lens, P, 3, extra=2)
    cache, d = L.alloc(pages), table.cuda()
    q, k, v, w = inputs(N, R, Hq, Hkv, D, dtype, 4)
    pos = torch.arange(R).int().repeat(N).cuda()
    f = (10000.0 ** (-torch.arange(0, D, 2) / D)).float().cuda()
    q, k = mqa.mqa_norm_rotate(q, k, *w, pos, f)
    length = torch.tensor(lens).int().cuda()
    zero = torch.zeros(N, dtype=torch.int32, device="cuda")
    mqa.mqa_kv_append(L, k, v, cache, d, zero, length)
    # the last 40 rows of each request look back
    last = torch.cat([torch.arange(i * R + n - 40, i * R + n) for i, n in enumerate(lens)]).cuda()
    rows, starts = q[last], torch.zeros(N * 40, dtype=torch.int32, device="cuda")
    ends = (pos[last] + 1).int()
    _, lse = mqa.mqa_attend_paged(L, rows, cache, d, starts, ends, return_lse=True)
    weights = torch.zeros(N, table.shape[1] * P, device="cuda")
    mqa.mqa_kv_weigh(L, rows, cache, d, starts, ends, lse, weights)
    want, tol = weigh_ref(pool_of(cache, L), rows.cpu(), table, starts.cpu(), ends.cpu(), lse.cpu())
    assert ref.differs(weights, want, tol + 2.0 ** -24 * want) == 0
    # cut: the kept positions' attention is what the list gave, of the values that stand there
    kept = torch.empty_like(weights)
    listed, count = mqa.mqa_kv_select(weights, length, 200, 4, 50, kept=kept)
    mqa.mqa_kv_keep(L, cache, d, listed, count)
    q1 = q[last[39::40]].contiguous()
    out, lse1 = mqa.mqa_attend_paged(L, q1, cache, d, zero, count, return_lse=True)
    seen = torch.arange(256)[None] < count.cpu()[:, None]
    want, wlse, tol, tol_lse = serve_ref.attend(pool_of(cache, L), q1.cpu(), table, seen)
    assert ref.differs(out, want, tol) == 0 and ref.differs(lse1, wlse, tol_lse) == 0
    # the next token: stored behind what was kept, its weight on top of the kept weights
    q2, k2, v2, w2 = inputs(N, 1, Hq, Hkv, D, dtype, 5)
    q2, k2 = mqa.mqa_norm_rotate(q2, k2, *w, length, f)
    mqa.mqa_kv_append(L, k2, v2, cache, d, count)
    out, lse2 = mqa.mqa_attend_paged(L, q2, cache, d, zero, count + 1, return_lse=True)
    before = kept.clone()
    mqa.mqa_kv_weigh(L, q2, cache, d, zero, count + 1, lse2, kept)
    added, tol = weigh_ref(pool_of(cache, L), q2.cpu(), table, zero.cpu(), count.cpu() + 1, lse2.cpu())
    total = before.cpu().double() + added
    assert ref.differs(kept, total, tol + 2.0 ** -23 * total) == 0


@pytest.mark.parametrize("D,P,B,codes", [(128, 64, 64, "e4m3"), (64, 16, 16, "int8")])
def test_a_tree_is_verified_and_its_path_moved(D, P, B, codes):
    say(f"case: tree, then its path {D} {P} {B} {codes}")
    Hq, Hkv, dtype, lens, R = 8, 2, BF16, [333, 90], 7
    L = mqa.KVLayout(Hkv, D, P, B, codes)
    table, pages = ref.make_table([n + R for n in lens], P, 6)
    cache, d = L.alloc(pages), table.cuda()
    q, k, v, w = inputs(2, max(lens), Hq, Hkv, D, dtype, 7)
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    length = torch.tensor(lens).int().cuda()
    mqa.mqa_kv_append(L, k, v, cache, d, zero, length)
    parents, path = (-1, -1, 0, 0, 1, 2, 4), (1, 4, 6)
    see = torch.zeros(R, R, dtype=torch.bool)
    for t, parent in enumerate(parents):
        if parent >= 0:
            see[t] = see[parent]
        see[t, t] = True
    q, k, v, w = inputs(2, R, Hq, Hkv, D, dtype, 8)
    mqa.mqa_kv_append(L, k, v, cache, d, length)
    ends, starts = length.repeat_interleave(R), torch.zeros(2 * R, dtype=torch.int32, device="cuda")
    bits = see.repeat(2, 1)
    out = mqa.mqa_attend_tree(L, q, cache, d, starts, ends, serve_ref.words(bits).cuda())
    seen = serve_ref.tree_seen(starts.cpu(), ends.cpu(), serve_ref.words(bits), table.shape[1] * P)
    want, _, tol, _ = serve_ref.attend(pool_of(cache, L), q.cpu(), table, seen)
    assert ref.differs(out, want, tol) == 0
    listed = (length[:, None] + torch.tensor(path, device="cuda")).int()
    mqa.mqa_kv_keep(L, cache, d, listed, torch.full_like(length, 3), length)
    # each accepted token over the chain that now stands there
    rows = torch.tensor([i * R + t for i in range(2) for t in path])
    ends = (length.cpu()[:, None] + 1 + torch.arange(3)).view(-1).int()
    got = mqa.mqa_attend_paged(L, q[rows.cuda()], cache, d, starts[:6], ends.cuda())
    chain = torch.arange(table.shape[1] * P)[None] < ends[:, None]
    want, _, tol, _ = serve_ref.attend(pool_of(cache, L), q.cpu()[rows], table, chain)
    assert ref.differs(got, want, tol) == 0


def test_a_captured_step_replays_as_requests_grow():
    Hq, Hkv, D, P, N = 8, 2, 128, 16, 3
    L = mqa.KVLayout(Hkv, D, P, P, "e4m3")
    table, pages = ref.make_table([400] * N, P, 9)
    d = table.cuda()
    f = (10000.0 ** (-torch.arange(0, D, 2) / D)).float().cuda()
    x = torch.empty(N, Hq + 2 * Hkv, D, dtype=BF16, device="cuda")
    w = [torch.ones(D, dtype=BF16, device="cuda")] * 2
    zero = torch.zeros(N, dtype=torch.int32, device="cuda")
    work = torch.empty(mqa.workspace_size_attend(N, 1, Hq, L, table.shape[1] * P), dtype=torch.uint8,
                       device="cuda")

    def step(cache, at, weights):
        q, k = mqa.mqa_norm_rotate(x[:, :Hq], x[:, Hq:Hq + Hkv], *w, at, f)
        mqa.mqa_kv_append(L, k, x[:, Hq + Hkv:], cache, d, at)
        out, lse = mqa.mqa_attend_paged(L, q, cache, d, zero, at + 1, return_lse=True, workspace=work)
        mqa.mqa_kv_weigh(L, q, cache, d, zero, at + 1, lse, weights)
        near = mqa.mqa_attend_window(L, q, cache, d, zero, at + 1, 50, 4, workspace=work)
        listed, count = mqa.mqa_kv_select(weights, at + 1, 100, 4, 20)
        mqa.mqa_kv_keep(L, cache, d, listed, count)
        return out, near, listed, count

    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    state = [(L.alloc(pages), torch.tensor([90, 99, 3]).int().cuda(), torch.zeros(N, table.shape[1] * P, device="cuda"))
             for _ in range(2)]
    x.normal_(generator=g)
    step(*state[0])
    for t in state[0][0], state[0][2]:
        t.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(*state[0])
    for i in range(4):
        x.normal_(generator=g)
        graph.replay()
        eager = step(*state[1])
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert torch.equal(a, b), i
        assert torch.equal(state[0][0], state[1][0]) and torch.equal(state[0][2], state[1][2])
        for s in state:
            s[1].add_(7)


def test_bounded_cache_example():
    say("case: examples/bounded_cache.py")
    import bounded_cache

    assert bounded_cache.main(["--prompt", "700", "--chunk", "300", "--keep", "256", "--requests", "2"]) == 0


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (12, 12, 64), (64, 1, 128)])
def test_the_largest_batch_s_workspaces_serve_smaller_ones(Hq, Hkv, D):
    L = mqa.KVLayout(Hkv, D)
    from fp8_mqa_logits_amd import attend as A
    lib = A._load()
    for requests, R, positions in ((512, 1, 131072), (96, 7, 20000), (1, 4096, 49152), (3, 700, 1 << 20)):
        weigh = mqa.workspace_size_weigh(requests, R, Hq, L, positions)
        attend = mqa.workspace_size_attend(requests, R, Hq, L, positions)
        for n in sorted({1, 2, 5, 31, 95, 300, requests}):
            for r in sorted({1, 2, 4, 16, 33, 100, 333, R}):
                for p in (64, 777, 4096, 19999, positions):
                    if n > requests or r > R or p > positions:
                        continue
                    assert 0 < mqa.workspace_size_weigh(n, r, Hq, L, p) <= weigh, (n, r, p)
                    for kind in (2, 3):
                        need = lib.workspace_size_attend_call(n, r, Hq, Hkv, D, p, kind, 0)
                        assert 0 < need <= attend, (n, r, p, kind)
    assert lib.workspace_size_attend_call(1, 1, Hq, Hkv, D, 100, 4, 0) == 0
