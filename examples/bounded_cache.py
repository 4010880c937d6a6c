"""Serving with a cache of bounded length, on one GPU: queries and keys are normed and
rotated, prompts go into the paged 8-bit cache chunk by chunk while every position
collects the attention weight it receives, the cache is cut to the heaviest positions, and
decoding goes on from there, with a tree of drafted tokens a step of which one path is
accepted. A second layer of the same tokens sees a sliding window with sinks, and its
pages in between are given back.

    python examples/bounded_cache.py [--prompt 1500] [--keep 512] [--requests 3] [--steps 4]

Synthetic data and random weights. The numbers printed: the share of the attention weight
that the kept positions hold, and how far the attention over them is from the attention
over the same positions before they were moved.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_mqa_logits_amd as mqa  # noqa: E402

HEADS, KV_HEADS, DIM, PAGE = 32, 8, 128, 16
WINDOW, SINKS = 200, 4
# a tree of seven drafts: the parent of each (-1: the context), and the paths through it
PARENTS = (-1, -1, 0, 0, 1, 2, 4)
PATHS = ((0, 2, 5), (1, 4, 6), (0, 3))


def ints(values, device):
    return torch.as_tensor(values, dtype=torch.int32, device=device)


def tree_mask():
    """[drafts] int: bit x of word t is set where draft t sees draft x."""
    see = []
    for t, parent in enumerate(PARENTS):
        see.append((1 << t) | (see[parent] if parent >= 0 else 0))
    return see


class Layer:
    """Random projections of a hidden state to rotated queries and keys, and values."""

    def __init__(self, hidden, gen, device):
        self.qkv = (torch.randn(hidden, (HEADS + 2 * KV_HEADS) * DIM, generator=gen, device=device)
                    / hidden ** 0.5).bfloat16()
        self.weights = [(1 + 0.1 * torch.randn(DIM, generator=gen, device=device)).bfloat16()
                        for _ in range(2)]
        i = torch.arange(0, DIM, 2, device=device)
        self.inv_freq = 10000.0 ** (-i.float() / DIM)

    def project(self, x, positions):
        qkv = (x.bfloat16() @ self.qkv).view(-1, HEADS + 2 * KV_HEADS, DIM)
        q, k, v = qkv.split([HEADS, KV_HEADS, KV_HEADS], 1)
        q, k = mqa.mqa_norm_rotate(q, k, *self.weights, positions, self.inv_freq)
        return q, k, v


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--prompt", type=int, default=1500)
    ap.add_argument("--chunk", type=int, default=512)
    ap.add_argument("--keep", type=int, default=512)
    ap.add_argument("--requests", type=int, default=3)
    ap.add_argument("--steps", type=int, default=4)
    a = ap.parse_args(argv)
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(11)
    hidden, N, drafts = 256, a.requests, len(PARENTS)
    layer = Layer(hidden, gen, dev)
    layout = mqa.KVLayout(KV_HEADS, DIM, page_size=PAGE, block=PAGE)
    pages = -(-(a.prompt + (a.steps + 1) * (drafts + 1)) // PAGE)
    table = torch.randperm(N * pages, generator=gen, device=dev).int().view(N, pages)
    cache, windowed = layout.alloc(N * pages, dev), layout.alloc(N * pages, dev)
    window_table = table.clone()
    weights = torch.zeros(N, pages * PAGE, device=dev)

    # the prompts, a chunk of every request at a time
    for first in range(0, a.prompt, a.chunk):
        n = min(a.chunk, a.prompt - first)
        positions = first + torch.arange(n, dtype=torch.int32, device=dev).repeat(N)
        q, k, v = layer.project(torch.randn(N * n, hidden, generator=gen, device=dev), positions)
        at = ints([first] * N, dev)
        for c in (cache, windowed):
            mqa.mqa_kv_append(layout, k, v, c, table, at)
        starts, ends = torch.zeros_like(positions), positions + 1
        out, lse = mqa.mqa_attend_paged(layout, q, cache, table, starts, ends, return_lse=True)
        mqa.mqa_kv_weigh(layout, q, cache, table, starts, ends, lse, weights)
        mqa.mqa_attend_window(layout, q, windowed, window_table, starts, ends, WINDOW, SINKS)
    heads = float(weights.sum()) / (N * a.prompt)
    print(f"{N} x {a.prompt} tokens: a row hands out {heads:.4f} of weight over its {HEADS} heads")

    # the cache is cut; what the second layer's windows have left behind is given back
    length = ints([a.prompt] * N, dev)
    kept = torch.empty_like(weights)
    chosen, count = mqa.mqa_kv_select(weights, length, a.keep, SINKS, a.keep // 4, kept=kept)
    probe = q.view(N, -1, HEADS, DIM)[:, -1].contiguous()  # the last rows of the prompts
    zero = ints([0] * N, dev)
    before = mqa.mqa_attend_topk(layout, probe, cache, table, chosen, zero, length)
    share = float((kept.sum() / weights.sum()).item())
    mqa.mqa_kv_keep(layout, cache, table, chosen, count)
    after = mqa.mqa_attend_paged(layout, probe, cache, table, zero, count)
    off = float((after.float() - before.float()).norm() / before.float().norm())
    print(f"kept {a.keep} positions with {share:.3f} of the weight; attention over them, moved, is "
          f"off by {off:.1e}")
    weights, kept = kept, weights
    gone = slice(-(-SINKS // PAGE), max(-(-SINKS // PAGE), (a.prompt - WINDOW) // PAGE))
    window_table[:, gone] = -1

    # decoding: a tree of drafts behind every cache, of which one path stays
    mask = ints(tree_mask(), dev).repeat(N)[:, None].contiguous()
    depth = [0] * drafts
    for t, parent in enumerate(PARENTS):
        depth[t] = 0 if parent < 0 else depth[parent] + 1
    seen = a.prompt  # tokens so far, which positions go by
    for step in range(a.steps):
        positions = ints([seen + d for d in depth] * N, dev)
        q, k, v = layer.project(torch.randn(N * drafts, hidden, generator=gen, device=dev), positions)
        mqa.mqa_kv_append(layout, k, v, cache, table, count)
        ends = count.repeat_interleave(drafts)
        out = mqa.mqa_attend_tree(layout, q, cache, table, torch.zeros_like(ends), ends, mask)
        assert bool(torch.isfinite(out.float()).all())
        path = PATHS[step % len(PATHS)]
        mqa.mqa_kv_keep(layout, cache, table, count[:, None] + ints([path], dev), ints([len(path)] * N, dev),
                        count)
        # the accepted tokens' rows hand out their weight, and go on in the second layer
        rows = (torch.arange(N, device=dev)[:, None] * drafts + ints([path], dev)).view(-1)
        starts = torch.zeros_like(rows, dtype=torch.int32)
        ends = (count[:, None] + 1 + torch.arange(len(path), device=dev)).view(-1).int()
        _, lse = mqa.mqa_attend_paged(layout, q[rows], cache, table, starts, ends, return_lse=True)
        mqa.mqa_kv_weigh(layout, q[rows], cache, table, starts, ends, lse, weights)
        mqa.mqa_kv_append(layout, k[rows], v[rows], windowed, window_table, ints([seen] * N, dev))
        ends = ints([seen + 1 + i for i in range(len(path))] * N, dev)
        out = mqa.mqa_attend_window(layout, q[rows], windowed, window_table, starts, ends, WINDOW, SINKS)
        assert bool(torch.isfinite(out.float()).all())
        count, seen = count + len(path), seen + len(path)
    print(f"{a.steps} trees of {drafts} drafts: {seen - a.prompt} tokens accepted, caches hold "
          f"{count.tolist()} of {seen} positions")
    return 0


if __name__ == "__main__":
    sys.exit(main())
