"""Sparse attention of one layer, end to end on one GPU: a prompt's keys and
values go into the paged 8-bit cache chunk by chunk, the FP8 indexer picks each
row's top-k positions, attention reads those; then a few tokens are decoded the
same way for a batch of requests.

    python examples/sparse_attention.py [--prompt 3000] [--requests 4] [--tokens 8]

Synthetic data and random weights. Rows that see at most k positions list all
of them, so that for these the listed attention has to give what attention over
the whole range gives; the largest difference is printed (and checked).
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_mqa_logits_amd as mqa  # noqa: E402
import mqa_workloads as W  # noqa: E402

TOPK, PAGE = 512, 64
HEADS, KV_HEADS, DIM = 32, 4, 128


class Layer:
    """Random projections of a hidden state to what the layer's attention and
    its indexer take."""

    def __init__(self, hidden, gen, device):
        def weight(n):
            return torch.randn(hidden, n, generator=gen, device=device) / hidden ** 0.5

        self.qkv = weight((HEADS + 2 * KV_HEADS) * DIM).bfloat16()
        self.index_q, self.index_w = weight(W.HEADS * W.DIM), weight(W.HEADS)

    def project(self, x):
        """(q, k, v, index q, index weights) of rows x [rows, hidden]; q, k and
        v are slices of one product."""
        rows = x.shape[0]
        qkv = (x.bfloat16() @ self.qkv).view(rows, HEADS + 2 * KV_HEADS, DIM)
        q, k, v = qkv.split([HEADS, KV_HEADS, KV_HEADS], 1)
        iq = (x @ self.index_q).view(rows, W.HEADS, W.DIM).to(torch.float8_e4m3fn)
        return q, k, v, iq, (x @ self.index_w) / W.HEADS ** 0.5


def ints(values, device):
    return torch.as_tensor(values, dtype=torch.int32, device=device)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--prompt", type=int, default=3000)
    ap.add_argument("--chunk", type=int, default=1024)
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=8)
    a = ap.parse_args(argv)
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(7)
    hidden = 256
    layer = Layer(hidden, gen, dev)
    layout = mqa.KVLayout(KV_HEADS, DIM, page_size=PAGE, block=PAGE)

    # both caches: the same page numbers, each request its own pages
    most = a.prompt + a.tokens
    pages = -(-most // PAGE)
    table = torch.randperm(a.requests * pages, generator=gen, device=dev).int().view(a.requests, pages)
    cache = layout.alloc(a.requests * pages, dev)
    index_cache = torch.empty(a.requests * pages, PAGE * (W.DIM + 4), dtype=torch.uint8, device=dev)
    for i in range(a.requests):
        rng = np.random.default_rng(i)
        keys = W.encode_e4m3(rng.standard_normal((pages * PAGE, W.DIM)))
        scales = W.ue8m0_bytes(rng.integers(-4, 1, pages * PAGE))
        made, order = W.paged_cache(keys, scales, PAGE, spare_pages=0)
        index_cache[table[i].long()] = torch.from_numpy(made[order]).to(dev)

    worst = 0.0
    # the prompts, a request and a chunk at a time
    for i in range(a.requests):
        for first in range(0, a.prompt, a.chunk):
            n = min(a.chunk, a.prompt - first)
            q, k, v, iq, iw = layer.project(torch.randn(n, hidden, generator=gen, device=dev))
            mqa.mqa_kv_append(layout, k, v, cache, table[i], ints([first], dev))
            starts = torch.zeros(n, dtype=torch.int32, device=dev)
            ends = first + 1 + torch.arange(n, dtype=torch.int32, device=dev)
            picked = mqa.mqa_topk_prefill_paged(iq, index_cache, table[i], PAGE, first + n, iw,
                                                starts, ends, TOPK)
            out = mqa.mqa_attend_topk(layout, q, cache, table[i], picked, starts, ends)
            if first < TOPK:  # rows whose list is everything they see
                every = min(TOPK - first, n)
                full = mqa.mqa_attend_paged(layout, q[:every], cache, table[i], starts[:every],
                                            ends[:every])
                worst = max(worst, float((full.float() - out[:every].float()).abs().max()))
    print(f"prompts: {a.requests} x {a.prompt} tokens, largest difference where the list is "
          f"everything: {worst:.2e}")
    # bf16 outputs of order 1: half a last place and the reordered fp32 sums
    assert worst < 2.0 ** -6

    # decoding, all requests together
    for t in range(a.tokens):
        at = a.prompt + t
        q, k, v, iq, iw = layer.project(torch.randn(a.requests, hidden, generator=gen, device=dev))
        mqa.mqa_kv_append(layout, k, v, cache, table, ints([at] * a.requests, dev))
        starts, ends = ints([0] * a.requests, dev), ints([at + 1] * a.requests, dev)
        picked = mqa.mqa_topk_decode_paged(iq, index_cache, table, PAGE, iw, starts, ends, TOPK, 1)
        out, lse = mqa.mqa_attend_topk(layout, q, cache, table, picked, starts, ends,
                                       return_lse=True)
    if a.tokens:
        whole, all_lse = mqa.mqa_attend_paged(layout, q, cache, table, starts, ends,
                                              return_lse=True)
        share = torch.exp(lse - all_lse).mean().item()
        print(f"decoded {a.tokens} x {a.requests} tokens; the last ones' {TOPK} listed positions "
              f"hold {share:.3f} of the softmax over all {at + 1}")
        assert 0.0 < share <= 1.0 + 1e-5 and bool(torch.isfinite(out.float()).all())
    # what was stored, read back: the last token's values, rounded to 8 bits
    back, _ = mqa.mqa_kv_read(layout, cache, table, ints([most - 1] * a.requests, dev), None, 1)
    off = float((back.float() - k.float()).norm() / k.float().norm()) if a.tokens else 0.0
    print(f"stored keys against their bf16 originals: {off:.3f} relative")
    assert off < 0.06
    return 0


if __name__ == "__main__":
    sys.exit(main())
