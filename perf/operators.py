"""Cases of the operators on the paged 8-bit key/value cache: attention over
each row's range of positions, attention over each row's listed positions (the
indexer's top-k output), and storing new tokens and reading them back.

The cache. A page holds P tokens: codes [2][kv_heads][P][D] (keys, then
values; e4m3 or int8 bytes), then fp32 scales [2][kv_heads][P / B] (one for
each block of B tokens and head), padded to a multiple of 128 bytes. Position
j of request i is slot j % P of page table[i, j // P]. Row r belongs to
request r // R.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one user typing: a single request's next token, latency counts
        attend("decode_1x1_777", N=1, R=1, ctx=777, Hq=32, Hkv=8),
        # a serving batch of uneven contexts, small pages, int8 cache
        attend("decode_48x1_ragged", N=48, R=1, ctx=20011, Hq=32, Hkv=4, P=16, B=16, type="fp16",
               codes="int8", ragged=True),
        # long contexts in the cache, a token each: the cache's bytes count
        attend("decode_32x1_131072", N=32, R=1, ctx=131072, Hq=16, Hkv=2),
        # four speculative rows a request, an odd group of heads, narrow heads
        attend("verify_24x4_ragged", N=24, R=4, ctx=9001, Hq=40, Hkv=8, D=64, P=32, B=32,
               ragged=True),
        # a short prompt under a sliding window, one key head per query head,
        # with padding rows that see nothing
        attend("window_333", N=1, R=333, ctx=333, Hq=12, Hkv=12, D=64, type="fp16", codes="int8",
               see="window", pad=True),
        # the chunk of two requests of the second benchmark configuration
        attend("packed_2048x32768", N=1, R=2048, ctx=32768, Hq=32, Hkv=8, see="packed"),
        # a long prompt's chunk at the end of its context: matrix work counts
        attend("chunk_4096x49152", N=1, R=4096, ctx=49152, Hq=32, Hkv=4),
        # the next token of a few requests over the indexer's 512 positions
        listing("topk_8x1_512", N=8, R=1, ctx=30000, Hq=32, Hkv=8, k=512),
        # two speculative rows of many requests over 2048 positions
        listing("topk_64x2_2048", N=64, R=2, ctx=65536, Hq=32, Hkv=8, k=2048, type="fp16"),
        # a prompt's chunk, each row with its own 2048 positions, all query
        # heads on one key head
        listing("topk_chunk_4096_2048", N=1, R=4096, ctx=65536, Hq=64, Hkv=1, k=2048),
        # a decode step's new tokens, each into a partly filled block
        storing("store_64x1", N=64, R=1, first=20011, Hkv=8),
        # a prompt's chunk stored and handed over
        storing("store_16384", N=1, R=16384, first=16384, Hkv=8),
    ]


HEADS = [(32, 8), (32, 4), (16, 2), (40, 8), (12, 12), (28, 4), (8, 1), (64, 1)]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["decode", "decode", "prefill", "topk", "topk", "store"])
    Hq, Hkv = rng.choice(HEADS)
    P = rng.choice([16, 32, 64, 128])
    more = {"D": rng.choice([64, 128, 128]), "P": P, "B": rng.choice([b for b in (16, 32, 64) if b <= P]),
            "type": rng.choice(["bf16", "fp16"]), "codes": rng.choice(["e4m3", "e4m3", "int8"])}
    if kind == "store":
        N = log_int(1, 256)
        return storing(None, N=N, R=log_int(1, max(1, 16384 // N)), first=log_int(1, 32768), Hkv=Hkv,
                       **(more | {"type": rng.choice(["bf16", "fp16", "fp32"])}))
    if kind == "topk":
        N, R = (1, log_int(64, 4096)) if rng.random() < 0.4 else (log_int(1, 96), rng.randint(1, 4))
        k = rng.choice([512, 1024, 2048])
        k = max(64, min(k, 4096 * 2048 * 64 // (N * R * Hq), 4096 * 2048 * 2 // (N * R * Hkv)))
        return listing(None, N=N, R=R, ctx=log_int(200, 65536), Hq=Hq, Hkv=Hkv, k=k,
                       ragged=rng.random() < 0.5, **more)
    if kind == "prefill":
        R = log_int(16, 4096)
        ctx = log_int(R, 45000)
        Hq, Hkv = rng.choice([h for h in HEADS if h[0] <= 32])
        see = rng.choice(["causal", "causal", "packed", "window", "full"])
        return attend(None, N=1, R=R, ctx=ctx, Hq=Hq, Hkv=Hkv, see=see, pad=rng.random() < 0.3,
                      **more)
    N, R = log_int(1, 96), rng.choice([1, 1, 1, 2, 4, 7])
    most = min(131072, 32 * 131072 * 2 // (N * Hkv))  # no more bytes than the largest listed
    return attend(None, N=N, R=R, ctx=log_int(1, most), Hq=Hq, Hkv=Hkv, ragged=rng.random() < 0.6,
                  pad=rng.random() < 0.2, **more)


def attend(name, N, R, ctx, Hq, Hkv, D=128, P=64, B=64, type="bf16", codes="e4m3", see="causal",
           ragged=False, pad=False):
    case = {"op": "paged", "N": N, "R": R, "ctx": ctx, "Hq": Hq, "Hkv": Hkv, "D": D, "P": P,
            "B": B, "type": type, "codes": codes, "see": see, "ragged": ragged, "pad": pad}
    return case if name is None else {"name": name, **case}


def listing(name, N, R, ctx, Hq, Hkv, k, D=128, P=64, B=64, type="bf16", codes="e4m3",
            ragged=False):
    case = {"op": "topk", "N": N, "R": R, "ctx": ctx, "Hq": Hq, "Hkv": Hkv, "D": D, "P": P, "B": B,
            "type": type, "codes": codes, "see": "causal", "ragged": ragged, "pad": False, "k": k}
    return case if name is None else {"name": name, **case}


def storing(name, N, R, first, Hkv, D=128, P=64, B=64, type="bf16", codes="e4m3"):
    case = {"op": "store", "N": N, "R": R, "first": first, "Hkv": Hkv, "D": D, "P": P, "B": B,
            "type": type, "codes": codes}
    return case if name is None else {"name": name, **case}


# ---------------------------------------------------------------- the inputs

def lengths(case):
    """Each request's context length: a fact of the case, not of the seed."""
    if case["op"] == "store":
        r = random.Random(case["N"] * 7919 + case["first"])
        return [r.randint(0, case["first"]) if i else case["first"] for i in range(case["N"])]
    r = random.Random(case["N"] * 7919 + case["ctx"])
    low = max(1, case["R"], case["ctx"] // 8)
    return [r.randint(min(low, case["ctx"]), case["ctx"]) if case["ragged"] and i else case["ctx"]
            for i in range(case["N"])]


def ranges(case):
    """(starts, ends) of the rows, two int64 tensors on the CPU."""
    R, ctx = case["R"], case["ctx"]
    t = torch.arange(R).repeat(case["N"])
    length = torch.tensor(lengths(case)).repeat_interleave(R)
    ends = length - (R - 1 - t)
    starts = torch.zeros_like(ends)
    if case["see"] == "packed":  # two requests in one key numbering, half the rows each
        half, base = R // 2, (ctx // 2) // case["P"] * case["P"]
        first = t < half
        starts = torch.where(first, 0, base)
        ends = torch.where(first, base - (half - 1 - t), ctx - (R - 1 - t))
    elif case["see"] == "window":
        starts = (ends - max(1, ctx // 4)).clamp(min=0)
    elif case["see"] == "full":
        ends = length.clone()
    if case["pad"]:  # a batch filled up with rows that see nothing
        starts[-(R // 8 + 1):] = 0
        ends[-(R // 8 + 1):] = 0
    ends = torch.maximum(ends.clamp(min=0), starts)
    return starts, ends


def page_bytes(case):
    n = 2 * case["Hkv"] * (case["P"] * case["D"] + case["P"] // case["B"] * 4)
    return (n + 127) // 128 * 128


def power_of_two_scale(amax, codes):
    """The smallest 2^e >= 2^-126 with amax <= M * 2^e, in 32 bits."""
    top, shift = (0.875, 9) if codes == "e4m3" else (127 / 128, 7)  # M = top * 2^shift
    m, e = torch.frexp(amax)
    return torch.ldexp(torch.ones_like(amax), (e - shift + (m > top).int()).clamp(min=-126))


def to_codes(x, codes):
    """fp32 values already divided by their scale -> code bytes."""
    if codes == "e4m3":
        return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)


def from_codes(c, codes):
    return c.view(torch.float8_e4m3fn if codes == "e4m3" else torch.int8).float()


def make_cache(case, num_pages, gen):
    """A pool of pages full of tokens: Gaussian keys with a few loud channels
    and values, tokens of uneven loudness, each block scaled by its largest."""
    Hkv, P, D, B = case["Hkv"], case["P"], case["D"], case["B"]
    cache = torch.zeros(num_pages, page_bytes(case), dtype=torch.uint8, device=DEVICE)
    loud = torch.ones(2, Hkv, 1, D, device=DEVICE)
    loud[0, :, :, torch.randperm(D, generator=gen, device=DEVICE)[:4]] = 4.0
    step = max(1, (1 << 28) // (2 * Hkv * P * D))
    for a in range(0, num_pages, step):
        n = min(step, num_pages - a)
        x = torch.randn(n, 2, Hkv, P, D, generator=gen, device=DEVICE).mul_(loud)
        x.mul_(torch.exp2(torch.randn(n, 2, Hkv, P, 1, generator=gen, device=DEVICE) * 0.5))
        x = x.view(n, 2, Hkv, P // B, B * D)
        s = power_of_two_scale(x.abs().amax(-1, keepdim=True), case["codes"])
        cache[a:a + n, :2 * Hkv * P * D] = to_codes(x.div_(s), case["codes"]).view(n, -1)
        cache[a:a + n, 2 * Hkv * P * D:][:, :2 * Hkv * (P // B) * 4] = s.view(n, -1).view(torch.uint8)
    return cache


def make_table(case, lens, gen):
    need = [-(-n // case["P"]) for n in lens]
    total, stride = sum(need), max(max(need), 1)
    perm = torch.randperm(total + 3, generator=gen, device=DEVICE).int()
    table = torch.full((len(lens), stride), -1, dtype=torch.int32, device=DEVICE)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    return table, total + 3


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    N, R, Hkv, D, dtype = case["N"], case["R"], case["Hkv"], case["D"], TYPES[case["type"]]
    lens = lengths(case)
    state = {"case": case, "layout": {"kv_heads": Hkv, "head_dim": D, "page_size": case["P"],
                                      "block": case["B"], "codes": case["codes"]}}
    if case["op"] == "store":
        state["table"], pages = make_table(case, [n + R for n in lens], gen)
        state["cache"] = make_cache(case, pages, gen)
        x = torch.randn(2, N * R, Hkv, D, generator=gen, device=DEVICE)
        x *= torch.exp2(torch.randn(2, N * R, Hkv, 1, generator=gen, device=DEVICE))
        state["k"], state["v"] = x[0].to(dtype), x[1].to(dtype)
        state["starts"] = torch.tensor(lens, dtype=torch.int32, device=DEVICE)
        # what is read back: the blocks that the new tokens fall into, from
        # each first block's start to the last new token
        state["from"] = state["starts"] // case["B"] * case["B"]
        state["count"] = state["starts"] + R - state["from"]
        return state
    state["table"], pages = make_table(case, lens, gen)
    state["cache"] = make_cache(case, pages, gen)
    # queries of a size that spreads a row's scores over a few units
    state["q"] = (torch.randn(N * R, case["Hq"], D, generator=gen, device=DEVICE) * 0.7).to(dtype)
    starts, ends = ranges(case)
    state["starts"] = starts.int().to(DEVICE)
    state["ends"] = ends.int().to(DEVICE)
    if case["op"] == "topk":
        state["indices"] = make_indices(case, starts.to(DEVICE), ends.to(DEVICE), gen)
    return state


def make_indices(case, starts, ends, gen):
    """Each row's k positions of largest index score (shared by the rows of a
    request in part, as an indexer's are), as position - start, -1 padded."""
    rows, k = case["N"] * case["R"], case["k"]
    span = max(int((ends - starts).max()), k)
    score = torch.rand(case["N"], 1, span, generator=gen, device=DEVICE).expand(-1, case["R"], -1)
    score = 0.7 * score.reshape(rows, span)
    score += 0.3 * torch.rand(rows, span, generator=gen, device=DEVICE)
    score.masked_fill_(torch.arange(span, device=DEVICE) >= (ends - starts)[:, None], -1.0)
    top = score.topk(k, dim=1, sorted=False)
    return torch.where(top.values >= 0, top.indices, -1).int()


# ------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        return run_own(state)
    return {"paged": plain_paged, "topk": plain_topk, "store": plain_store}[case["op"]](state)


def run_own(state):
    import fp8_mqa_logits_amd as mqa

    case = state["case"]
    layout = mqa.KVLayout(**state["layout"])
    if case["op"] == "paged":
        out, lse = mqa.mqa_attend_paged(layout, state["q"], state["cache"], state["table"],
                                        state["starts"], state["ends"], return_lse=True)
        return {"out": out, "lse": lse}
    if case["op"] == "topk":
        out, lse = mqa.mqa_attend_topk(layout, state["q"], state["cache"], state["table"],
                                       state["indices"], state["starts"], state["ends"],
                                       return_lse=True)
        return {"out": out, "lse": lse}
    mqa.mqa_kv_append(layout, state["k"], state["v"], state["cache"], state["table"],
                      state["starts"])
    k, v = mqa.mqa_kv_read(layout, state["cache"], state["table"], state["from"], state["count"],
                           case["R"] + case["B"] - 1, dtype=state["k"].dtype)
    return {"k": k, "v": v}


def softmax_sums(score, seen, v):
    """exp(score) over the seen positions times v, over its sum, and the
    logarithm of that sum; a row that sees nothing gives 0 and -inf."""
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return out, (top + torch.log(total)).squeeze(-1)


def split_pages(pages, case):
    """[..., page_bytes] -> codes [..., 2, Hkv, P, D], scales [..., 2, Hkv, P / B]."""
    Hkv, P, D, B = case["Hkv"], case["P"], case["D"], case["B"]
    n, lead = 2 * Hkv * P * D, pages.shape[:-1]
    codes = pages[..., :n].reshape(*lead, 2, Hkv, P, D)
    scales = pages[..., n:n + 2 * Hkv * (P // B) * 4].contiguous().view(torch.float32)
    return codes, scales.view(*lead, 2, Hkv, P // B)


def plain_paged(state):
    case, q = state["case"], state["q"]
    N, R, Hkv, D, B = case["N"], case["R"], case["Hkv"], case["D"], case["B"]
    G = case["Hq"] // Hkv
    codes, scales = split_pages(state["cache"][state["table"].clamp(min=0).long()], case)
    kv = from_codes(codes, case["codes"]) * scales.repeat_interleave(B, -1).unsqueeze(-1)
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, N, Hkv, -1, D)
    qs = q.float().view(N, R, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(N, Hkv, R * G, D)
    score = torch.matmul(qs, kv[0].transpose(-1, -2)) * (1.0 / math.sqrt(D))
    pos = torch.arange(kv.shape[3], device=q.device)
    seen = (pos >= state["starts"][:, None]) & (pos < state["ends"][:, None])
    seen = seen.view(N, 1, R, 1, -1).expand(-1, -1, -1, G, -1).reshape(N, 1, R * G, -1)
    out, lse = softmax_sums(score, seen, kv[1])
    out = out.view(N, Hkv, R, G, D).permute(0, 2, 1, 3, 4).reshape(N * R, Hkv * G, D)
    lse = lse.view(N, Hkv, R, G).permute(0, 2, 1, 3).reshape(N * R, Hkv * G)
    return {"out": out.to(q.dtype), "lse": lse}


def plain_topk(state):
    case, q, idx = state["case"], state["q"], state["indices"].long()
    N, R, Hkv, D, P, B = case["N"], case["R"], case["Hkv"], case["D"], case["P"], case["B"]
    rows, G = N * R, case["Hq"] // Hkv
    seen = idx >= 0
    pos = torch.where(seen, idx + state["starts"].long()[:, None], 0)
    request = torch.arange(rows, device=q.device)[:, None] // R
    page, slot = state["table"].long()[request, pos // P].clamp(min=0), pos % P
    n = 2 * Hkv * P * D
    codes, scales = split_pages(state["cache"], case)
    take = lambda w: (from_codes(codes[page, w, :, slot], case["codes"])  # noqa: E731
                      * scales[page, w, :, slot // B].unsqueeze(-1)).transpose(1, 2)
    score = torch.matmul(q.float().view(rows, Hkv, G, D), take(0).transpose(-1, -2))
    out, lse = softmax_sums(score * (1.0 / math.sqrt(D)), seen[:, None, None, :], take(1))
    return {"out": out.reshape(rows, Hkv * G, D).to(q.dtype), "lse": lse.reshape(rows, Hkv * G)}


def plain_store(state):
    case, cache, table = state["case"], state["cache"], state["table"].long()
    N, R, Hkv, D, P, B = case["N"], case["R"], case["Hkv"], case["D"], case["P"], case["B"]
    codes, kind = case["codes"], case["codes"]
    device, first = cache.device, state["starts"].long()
    blocks = (R - 1) // B + 2  # blocks of a request that its new tokens can fall into
    begin = first // B * B
    pos = begin[:, None] + torch.arange(blocks * B, device=device)  # [N, blocks * B]
    t = pos - first[:, None]
    old, new = t < 0, (t >= 0) & (t < R)
    live = old | new
    page = table.gather(1, (pos // P).clamp(max=table.shape[1] - 1)).clamp(min=0)
    slot = pos % P
    row = torch.arange(N, device=device)[:, None] * R + t.clamp(0, R - 1)
    n = 2 * Hkv * P * D
    pool = cache[:, :n].view(torch.uint8)
    at_codes = (torch.arange(2 * Hkv, device=device) * P * D)[:, None] + torch.arange(D, device=device)
    at_codes = slot[..., None, None] * D + at_codes  # byte of the page, [N, T, 2 * Hkv, D]
    scale_pool = cache[:, n:n + 2 * Hkv * (P // B) * 4]
    at_scale = torch.arange(2 * Hkv, device=device) * (P // B) + (slot // B)[..., None]
    at_scale = at_scale[..., None] * 4 + torch.arange(4, device=device)  # [N, T, 2 * Hkv, 4]
    was_scale = scale_pool[page[..., None, None], at_scale].view(torch.float32)
    was = from_codes(pool[page[..., None, None], at_codes], kind) * was_scale
    fresh = torch.stack((state["k"], state["v"]), 1).float()[row].view(N, -1, 2 * Hkv, D)
    value = torch.where(new[..., None, None], fresh, torch.where(old[..., None, None], was, 0.0))
    amax = torch.where(new[..., None, None], fresh.abs(), 0.0).amax(-1)
    amax = amax.view(N, blocks, B, 2 * Hkv).amax(2)
    scale = power_of_two_scale(amax, kind)
    keeps = old.view(N, blocks, B).any(2)[..., None]
    was_scale = was_scale.view(N, blocks, B, 2 * Hkv)[:, :, 0]
    scale = torch.where(keeps, torch.maximum(scale, was_scale), scale).repeat_interleave(B, 1)
    code = to_codes(value / scale[..., None], kind)
    page_live, n_, t_ = page[live][:, None, None], *live.nonzero(as_tuple=True)
    cache[page_live, at_codes[n_, t_]] = code[n_, t_]
    cache[page_live, n + at_scale[n_, t_]] = scale[n_, t_][..., None].contiguous().view(torch.uint8)
    value = from_codes(code, kind) * scale[..., None]
    value = torch.where(live[..., None, None], value, 0.0)[:, :R + B - 1].to(state["k"].dtype)
    value = value.reshape(N * (R + B - 1), 2, Hkv, D)
    return {"k": value[:, 0].contiguous(), "v": value[:, 1].contiguous()}


# ------------------------------------------------------- the work, and 64 bits

def work(case):
    """Each visible position's codes and scales once for a request and head,
    each query, output, list and table entry once; 4 D flops for each query
    head of a row and position it sees."""
    N, R, Hkv, D, B = case["N"], case["R"], case["Hkv"], case["D"], case["B"]
    token = 2 * Hkv * (D + 4 / B)
    if case["op"] == "store":
        size = 4 if case["type"] == "fp32" else 2
        back = sum(R + n - n // B * B for n in lengths(case))
        kept = back - N * R  # earlier tokens of partly filled blocks
        new = N * R * 2 * Hkv * D * size
        wide = N * (R + B - 1) * 2 * Hkv * D * size
        return {"bytes": new + kept * token + back * token + back * token + wide + 8 * N, "flops": 0}
    starts, ends = ranges(case)
    seen = (ends - starts).clamp(min=0)
    head = 2 * 2 * N * R * case["Hq"] * D + 4 * N * R * (case["Hq"] + 2)
    if case["op"] == "topk":
        seen = seen.clamp(max=case["k"])
        head += 4 * N * R * case["k"]
        lens = torch.tensor(lengths(case))
        tokens = int(torch.minimum(seen.view(N, R).sum(1), lens).sum())
    else:
        low = torch.where(seen > 0, starts, 1 << 30).view(N, R).amin(1)
        high = torch.where(seen > 0, ends, 0).view(N, R).amax(1)
        tokens = int((high - low).clamp(min=0).sum())
    return {"bytes": head + tokens * (token + 4 / case["P"]),
            "flops": 4 * D * case["Hq"] * int(seen.sum())}


def exact(case, seed):
    """The operators' definitions in 64 bits, a request, a head and a piece of
    the rows at a time."""
    s = prepare(case, seed)
    if case["op"] == "store":
        return exact_store(case, s)
    N, R, Hq, Hkv, D = case["N"], case["R"], case["Hq"], case["Hkv"], case["D"]
    G, P, B, kind = Hq // Hkv, case["P"], case["B"], case["codes"]
    value = grid_values(kind).to(DEVICE)
    out = torch.zeros(N * R, Hq, D, dtype=torch.float64, device=DEVICE)
    lse = torch.full((N * R, Hq), -math.inf, dtype=torch.float64, device=DEVICE)
    q64 = s["q"].double()
    table, starts, ends = s["table"].cpu(), s["starts"].cpu().tolist(), s["ends"].cpu().tolist()

    def tensor_of(pages, w, h):
        """[pages, P, D] values of keys (w = 0) or values (w = 1) of one head."""
        a = (w * Hkv + h) * P * D
        b = 2 * Hkv * P * D + (w * Hkv + h) * (P // B) * 4
        c = value[pages[:, a:a + P * D].long()].view(-1, P // B, B, D)
        x = pages[:, b:b + P // B * 4].contiguous().view(torch.float32).double()
        return (c * x[:, :, None, None]).view(-1, P, D)

    for i in range(N):
        need = -(-max([1] + ends[i * R:(i + 1) * R]) // P)
        pages = s["cache"][table[i, :need].long().to(DEVICE)]
        for h in range(Hkv):
            k = tensor_of(pages, 0, h).reshape(-1, D)
            v = tensor_of(pages, 1, h).reshape(-1, D)
            piece = max(1, (1 << 28) // (k.shape[0] * G if case["op"] == "paged" else case["k"] * D))
            for a in range(i * R, (i + 1) * R, piece):
                r = range(a, min(a + piece, (i + 1) * R))
                rows = slice(r.start, r.stop)
                x = q64[rows, h * G:(h + 1) * G]
                if case["op"] == "topk":
                    at = s["indices"][rows].long()
                    ok = at >= 0
                    at = torch.where(ok, at + s["starts"][rows].long()[:, None], 0)
                    z = (x @ k[at].transpose(1, 2)) / math.sqrt(D)
                    z = z.masked_fill(~ok[:, None], -math.inf)
                    lse[rows, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
                    out[rows, h * G:(h + 1) * G] = torch.nan_to_num(torch.softmax(z, -1)) @ v[at]
                    continue
                z = (x.reshape(-1, D) @ k.T).view(len(r), G, -1) / math.sqrt(D)
                at = torch.arange(k.shape[0], device=DEVICE)
                ok = (at >= s["starts"][rows, None]) & (at < s["ends"][rows, None])
                z.masked_fill_(~ok[:, None], -math.inf)
                lse[rows, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
                p = torch.nan_to_num(torch.softmax(z, -1))
                out[rows, h * G:(h + 1) * G] = (p.view(-1, k.shape[0]) @ v).view(len(r), G, D)
    return {"out": out, "lse": lse}


def grid_values(kind):
    """What each of the 256 codes stands for, in 64 bits."""
    c = torch.arange(256)
    if kind == "int8":
        return (c - 256 * (c >= 128)).double()
    e, m = (c >> 3) & 15, (c & 7).double()
    a = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2(e.double() - 7))
    return torch.where(c >= 128, -a, a)


def nearest(x, kind):
    """x rounded to what a code stands for: nearest, ties to even."""
    if kind == "int8":
        return torch.round(x)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def exact_store(case, s):
    N, R, Hkv, D, P, B = case["N"], case["R"], case["Hkv"], case["D"], case["P"], case["B"]
    kind, width = case["codes"], case["R"] + case["B"] - 1
    largest = 448.0 if kind == "e4m3" else 127.0
    value = grid_values(kind).to(DEVICE)
    k = torch.zeros(2, N, width, Hkv, D, dtype=torch.float64, device=DEVICE)
    table, firsts = s["table"].cpu(), s["starts"].cpu().tolist()
    x = torch.stack((s["k"], s["v"])).double().view(2, N, R, Hkv, D)
    for i in range(N):
        first, begin = firsts[i], firsts[i] // B * B
        kept = first - begin
        z = torch.zeros(2, -(-(kept + R) // B) * B, Hkv, D, dtype=torch.float64, device=DEVICE)
        z[:, kept:kept + R] = x[:, i]
        scale = z.view(2, -1, B, Hkv, D).abs().amax((2, 4)) / largest
        scale = torch.exp2(torch.ceil(torch.log2(scale.clamp(min=2.0 ** -126))))
        if kept:
            page = s["cache"][int(table[i, begin // P])]
            n, at = 2 * Hkv * P * D, begin % P
            c = value[page[:n].long()].view(2, Hkv, P, D)[:, :, at:at + kept]
            b = page[n:n + 2 * Hkv * (P // B) * 4].view(torch.float32).double()
            b = b.view(2, Hkv, P // B)[:, :, at // B]
            z[:, :kept] = (c * b[:, :, None, None]).transpose(1, 2)
            scale[:, 0] = torch.maximum(scale[:, 0], b)
        scale = scale.repeat_interleave(B, 1)[..., None]
        k[:, i, :kept + R] = (nearest(z / scale, kind) * scale)[:, :kept + R]
    k = k.view(2, N * width, Hkv, D)
    return {"k": k[0], "v": k[1]}
