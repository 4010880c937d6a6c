"""Cases of the operators around attention over the paged 8-bit key/value
cache: queries and keys normed and rotated before they go there, attention
through a sliding window with sinks and over trees of drafted tokens, and
eviction by accumulated attention weight (weighing, selecting, moving).

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
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one user's next token, far into a context: latency counts
        rotating("rotate_1", rows=1, first=777216, Hq=32, Hkv=8),
        # an odd prompt of a model with narrow heads, a quarter of them rotated, neighbours paired
        rotating("rotate_777_pairs", rows=777, first=0, Hq=28, Hkv=4, D=64, rot=16, pairs=True,
                 type="fp16"),
        # a prompt's chunk
        rotating("rotate_16384", rows=16384, first=49152, Hq=32, Hkv=8),
        # a serving batch of uneven contexts, each through its last 1024 tokens
        windowed("window_64x1_ragged", N=64, R=1, ctx=20011, Hq=32, Hkv=8, window=1024, sinks=4,
                 ragged=True),
        # a long prompt's chunk through a wide window, odd sizes
        windowed("window_4096x4095", N=1, R=4096, ctx=49152, Hq=32, Hkv=4, window=4095, sinks=5),
        # small trees of drafted tokens, narrow heads, int8 cache
        tree("tree_8x13_ragged", N=8, R=13, ctx=9001, Hq=40, Hkv=8, D=64, P=32, B=32, type="fp16",
             codes="int8", ragged=True),
        # large trees over long contexts
        tree("tree_16x64_32768", N=16, R=64, ctx=32768, Hq=32, Hkv=8),
        # a decode step of a batch adds to its positions' weights
        weighing("weigh_32x1_32768", N=32, R=1, ctx=32768, Hq=32, Hkv=8),
        # a prompt's chunk does
        weighing("weigh_2048x32768", N=1, R=2048, ctx=32768, Hq=32, Hkv=8),
        # a long prompt is cut to an eighth before it is decoded
        evicting("evict_1x65536_8192", N=1, ctx=65536, keep=8192, Hkv=8),
        # a batch of uneven contexts is cut to 2048 positions each, small pages
        evicting("evict_32x9001_2048", N=32, ctx=9001, keep=2048, Hkv=4, P=16, B=16, codes="int8",
                 type="fp16", ragged=True),
        # the accepted paths of drafted trees move together
        accepting("accept_64x13", N=64, R=13, first=20011, Hkv=8),
    ]


HEADS = [(32, 8), (32, 4), (16, 2), (40, 8), (12, 12), (28, 4), (8, 1)]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["rotate", "window", "window", "tree", "weigh", "weigh", "evict", "accept"])
    Hq, Hkv = rng.choice(HEADS)
    D, type = rng.choice([64, 128, 128]), rng.choice(["bf16", "fp16"])
    if kind == "rotate":
        return rotating(None, rows=log_int(1, 12000), first=rng.randint(0, 1000000), Hq=Hq, Hkv=Hkv,
                        D=D, rot=rng.choice([D, D, D // 2, 16]), pairs=rng.random() < 0.4, type=type)
    P = rng.choice([16, 32, 64, 128])
    more = {"D": D, "P": P, "B": rng.choice([b for b in (16, 32, 64) if b <= P]), "type": type,
            "codes": rng.choice(["e4m3", "e4m3", "int8"])}
    if kind == "window":
        N, R = (1, log_int(16, 3500)) if rng.random() < 0.5 else (log_int(1, 96), rng.randint(1, 4))
        return windowed(None, N=N, R=R, ctx=log_int(max(R, 50), 40000), Hq=Hq, Hkv=Hkv,
                        window=log_int(17, 4000), sinks=rng.choice([0, 1, 4, 4, 16, 33]),
                        ragged=rng.random() < 0.5, pad=rng.random() < 0.3, **more)
    if kind == "tree":
        N, R = log_int(1, 24), log_int(2, 64)
        return tree(None, N=N, R=R, ctx=log_int(1, min(32768, 400000 // N)), Hq=Hq, Hkv=Hkv,
                    ragged=rng.random() < 0.6, **more)
    if kind == "weigh":
        N, R = (1, log_int(8, 2000)) if rng.random() < 0.5 else (log_int(1, 32), rng.randint(1, 4))
        return weighing(None, N=N, R=R, ctx=log_int(max(R, 50), 30000), Hq=min(Hq, 32), Hkv=Hkv,
                        ragged=rng.random() < 0.5, pad=rng.random() < 0.3, **more)
    if kind == "evict":
        N = log_int(1, 32)
        ctx = log_int(300, min(65536, 500000 // N))
        return evicting(None, N=N, ctx=ctx, keep=max(64, min(log_int(ctx // 20 + 1, ctx), 65536 // N)),
                        Hkv=Hkv, ragged=rng.random() < 0.6, **more)
    return accepting(None, N=log_int(1, 128), R=log_int(2, 64), first=log_int(1, 32768), Hkv=Hkv, **more)


def named(name, case):
    return case if name is None else {"name": name, **case}


def rotating(name, rows, first, Hq, Hkv, D=128, rot=None, pairs=False, type="bf16"):
    return named(name, {"op": "rotate", "rows": rows, "first": first, "Hq": Hq, "Hkv": Hkv, "D": D,
                        "rot": D if rot is None else rot, "pairs": pairs, "type": type})


def windowed(name, N, R, ctx, Hq, Hkv, window, sinks, D=128, P=64, B=64, type="bf16", codes="e4m3",
             ragged=False, pad=False):
    return named(name, {"op": "window", "N": N, "R": R, "ctx": ctx, "Hq": Hq, "Hkv": Hkv, "D": D,
                        "P": P, "B": B, "type": type, "codes": codes, "ragged": ragged, "pad": pad,
                        "window": window, "sinks": sinks})


def tree(name, N, R, ctx, Hq, Hkv, D=128, P=64, B=64, type="bf16", codes="e4m3", ragged=False):
    return named(name, {"op": "tree", "N": N, "R": R, "ctx": ctx, "Hq": Hq, "Hkv": Hkv, "D": D,
                        "P": P, "B": B, "type": type, "codes": codes, "ragged": ragged, "pad": False})


def weighing(name, N, R, ctx, Hq, Hkv, D=128, P=64, B=64, type="bf16", codes="e4m3", ragged=False,
             pad=False):
    return named(name, {"op": "weigh", "N": N, "R": R, "ctx": ctx, "Hq": Hq, "Hkv": Hkv, "D": D,
                        "P": P, "B": B, "type": type, "codes": codes, "ragged": ragged, "pad": pad})


def evicting(name, N, ctx, keep, Hkv, D=128, P=64, B=64, type="bf16", codes="e4m3", ragged=False):
    return named(name, {"op": "evict", "N": N, "R": 1, "ctx": ctx, "keep": keep,
                        "sinks": min(4, keep // 4), "recent": keep // 4, "Hkv": Hkv, "D": D, "P": P,
                        "B": B, "type": type, "codes": codes, "ragged": ragged})


def accepting(name, N, R, first, Hkv, D=128, P=64, B=64, type="bf16", codes="e4m3"):
    return named(name, {"op": "accept", "N": N, "R": R, "ctx": first, "Hkv": Hkv, "D": D, "P": P,
                        "B": B, "type": type, "codes": codes, "ragged": True})


# ---------------------------------------------------------------- the inputs

def lengths(case):
    """Each request's context length: a fact of the case, not of the seed."""
    r = random.Random(case["N"] * 7919 + case["ctx"])
    low = min(max(1, case["R"], case["ctx"] // 8), case["ctx"])
    return [r.randint(low, case["ctx"]) if case["ragged"] and i else case["ctx"]
            for i in range(case["N"])]


def accepted(case):
    """How many drafted tokens of each request are accepted."""
    r = random.Random(case["N"] * 31 + case["R"])
    return [min(case["R"], r.randint(1, 1 + case["R"] // 2)) for _ in range(case["N"])]


def ends_of(case):
    """Causal ends of the rows, int64 on the CPU; padding rows end at 0."""
    t = torch.arange(case["R"]).repeat(case["N"])
    ends = torch.tensor(lengths(case)).repeat_interleave(case["R"]) - (case["R"] - 1 - t)
    if case["pad"]:  # a batch filled up with rows that see nothing
        ends[-(case["R"] // 8 + 1):] = 0
    return ends.clamp(min=0)


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


def make_tree(case, gen):
    """[N * R, words] int32: the drafts that a draft sees, itself and its
    ancestors; a draft's parent is one of the eight before it or the context."""
    N, R = case["N"], case["R"]
    back = torch.randint(1, 9, (N, R), generator=gen, device=DEVICE).cpu()
    see = torch.zeros(N, R, -(-R // 32) * 32, dtype=torch.bool)
    for t in range(R):
        parent = t - back[:, t]
        see[:, t] = torch.where((parent >= 0)[:, None], see[torch.arange(N), parent.clamp(min=0)], False)
        see[:, t, t] = True
    bits = see.view(N * R, -1, 32).long() << torch.arange(32)
    words = bits.sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).int().to(DEVICE)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    dtype, D, Hkv = TYPES[case["type"]], case["D"], case["Hkv"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEVICE)

    if case["op"] == "rotate":
        rows, Hq = case["rows"], case["Hq"]
        # q and k as they come: slices of one product with the values behind
        qkv = (normal(rows, Hq + 2 * Hkv, D) * torch.exp2(normal(rows, Hq + 2 * Hkv, 1))).to(dtype)
        i = torch.arange(0, case["rot"], 2, dtype=torch.float64, device=DEVICE)
        return {"case": case, "q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hkv],
                "q_weight": (1 + 0.2 * normal(D)).to(dtype), "k_weight": (1 + 0.2 * normal(D)).to(dtype),
                "positions": case["first"] + torch.arange(rows, dtype=torch.int32, device=DEVICE),
                "inv_freq": (500000.0 ** (-i / case["rot"])).float()}
    N, R = case["N"], case["R"]
    lens = lengths(case)
    state = {"case": case, "layout": {"kv_heads": Hkv, "head_dim": D, "page_size": case["P"],
                                      "block": case["B"], "codes": case["codes"]}}
    state["table"], pages = make_table(
        case, [n + (R if case["op"] in ("tree", "accept") else 0) for n in lens], gen)
    state["cache"] = make_cache(case, pages, gen)
    state["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEVICE)
    if case["op"] == "evict":
        # what attention leaves: a few heavy positions, many light ones
        shape = (N, state["table"].shape[1] * case["P"])
        w = torch.exp(normal(*shape) * 2 - 6)
        state["weights"] = torch.where(torch.arange(shape[1], device=DEVICE) < state["lens"][:, None], w, 0.0)
        state["kept"] = torch.empty_like(state["weights"])
        return state
    if case["op"] == "accept":
        count = torch.tensor(accepted(case), device=DEVICE)
        order = torch.rand(N, R, generator=gen, device=DEVICE).argsort(1)
        path = torch.where(torch.arange(R, device=DEVICE) < count[:, None], order, R).sort(1).values
        state["path"] = torch.where(path < R, path + state["lens"][:, None], -1).int()
        state["count"] = count.int()
        # what is read back: the blocks that the moved tokens fall into, from
        # each first block's start to the last of them
        state["from"] = state["lens"] // case["B"] * case["B"]
        state["back"] = state["lens"] + state["count"] - state["from"]
        return state
    # queries of a size that spreads a row's scores over a few units
    state["q"] = (normal(N * R, case["Hq"], D) * 0.7).to(dtype)
    if case["op"] == "tree":
        state["ends"] = state["lens"].repeat_interleave(R)
        state["mask"] = make_tree(case, gen)
    else:
        state["ends"] = ends_of(case).int().to(DEVICE)
    state["starts"] = torch.zeros_like(state["ends"])
    if case["op"] == "weigh":
        score, seen = scores(state)
        state["lse"] = torch.logsumexp(torch.where(seen, score, -math.inf), -1)
        state["lse"] = state["lse"].view(N, Hkv, R, -1).permute(0, 2, 1, 3).reshape(N * R, -1)
        # weights so far, of the size that this call adds
        state["weights"] = torch.rand(N, state["table"].shape[1] * case["P"], generator=gen, device=DEVICE)
        state["weights"] *= 2 * R * case["Hq"] / case["ctx"]
    return state


# ------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return run_own(state)
    return {"rotate": plain_rotate, "window": plain_window, "tree": plain_tree, "weigh": plain_weigh,
            "evict": plain_evict, "accept": plain_accept}[op](state)


def run_own(state):
    import fp8_mqa_logits_amd as mqa

    case, s = state["case"], state
    if case["op"] == "rotate":
        q, k = mqa.mqa_norm_rotate(s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"],
                                   s["inv_freq"], pairs=case["pairs"])
        return {"q": q, "k": k}
    layout = mqa.KVLayout(**s["layout"])
    if case["op"] == "window":
        out, lse = mqa.mqa_attend_window(layout, s["q"], s["cache"], s["table"], s["starts"], s["ends"],
                                         case["window"], case["sinks"], return_lse=True)
        return {"out": out, "lse": lse}
    if case["op"] == "tree":
        out, lse = mqa.mqa_attend_tree(layout, s["q"], s["cache"], s["table"], s["starts"], s["ends"],
                                       s["mask"], return_lse=True)
        return {"out": out, "lse": lse}
    if case["op"] == "weigh":
        return {"weights": mqa.mqa_kv_weigh(layout, s["q"], s["cache"], s["table"], s["starts"],
                                            s["ends"], s["lse"].contiguous(), s["weights"])}
    if case["op"] == "evict":
        listed, count = mqa.mqa_kv_select(s["weights"], s["lens"], case["keep"], case["sinks"],
                                          case["recent"], kept=s["kept"])
        mqa.mqa_kv_keep(layout, s["cache"], s["table"], listed, count)
        k, v = mqa.mqa_kv_read(layout, s["cache"], s["table"], torch.zeros_like(count), count,
                               case["keep"], dtype=TYPES[case["type"]])
        return {"listed": listed, "count": count, "kept": s["kept"], "k": k, "v": v}
    mqa.mqa_kv_keep(layout, s["cache"], s["table"], s["path"], s["count"], s["lens"])
    k, v = mqa.mqa_kv_read(layout, s["cache"], s["table"], s["from"], s["back"],
                           case["R"] + case["B"] - 1, dtype=TYPES[case["type"]])
    return {"k": k, "v": v}


def plain_rotate(state):
    case, rot = state["case"], state["case"]["rot"]
    angle = state["positions"].double()[:, None] * state["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turn(x, weight):
        y = x.float()
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * weight.float()
        part = y[..., :rot].unflatten(-1, (-1, 2) if case["pairs"] else (2, -1))
        axis = -1 if case["pairs"] else -2
        a, b = part.unbind(axis)
        part = torch.stack((a * cos - b * sin, b * cos + a * sin), axis).flatten(-2)
        return torch.cat((part, y[..., rot:]), -1).to(x.dtype)

    return {"q": turn(state["q"], state["q_weight"]), "k": turn(state["k"], state["k_weight"])}


def tokens(state, pos, which):
    """fp32 values [N, Hkv, T, D] of the positions [N, T] of every request."""
    case = state["case"]
    Hkv, P, D, B = case["Hkv"], case["P"], case["D"], case["B"]
    n = 2 * Hkv * P * D
    at = (pos // P).clamp(0, state["table"].shape[1] - 1)
    page, slot = state["table"].long().gather(1, at).clamp(min=0), pos % P
    codes = state["cache"][:, :n].view(-1, 2, Hkv, P, D)[page, which, :, slot]
    scale = state["cache"][:, n:n + 2 * Hkv * (P // B) * 4].view(torch.float32)
    scale = scale.view(-1, 2, Hkv, P // B)[page, which, :, slot // B]
    return (from_codes(codes, case["codes"]) * scale[..., None]).transpose(1, 2)


def products(state, pos):
    """Scores [N, Hkv, R * G, T] of the positions [N, T]."""
    case = state["case"]
    N, R, Hkv, D = case["N"], case["R"], case["Hkv"], case["D"]
    q = state["q"].float().view(N, R, Hkv, -1, D).transpose(1, 2).reshape(N, Hkv, -1, D)
    return torch.matmul(q, tokens(state, pos, 0).transpose(-1, -2).contiguous()) * (1.0 / math.sqrt(D))


def per_column(seen, state):
    """[N * R, T] or [N, R, T] -> [N, 1, R * G, T], as products() lays its columns out."""
    case = state["case"]
    N, R, G = case["N"], case["R"], case["Hq"] // case["Hkv"]
    return seen.view(N, 1, R, 1, -1).expand(-1, -1, -1, G, -1).reshape(N, 1, R * G, -1)


def scores(state):
    """Scores of every position, and which are seen: causal ranges."""
    case = state["case"]
    pos = torch.arange(state["table"].shape[1] * case["P"], device=DEVICE).expand(case["N"], -1)
    seen = (pos[0] >= state["starts"][:, None]) & (pos[0] < state["ends"][:, None])
    return products(state, pos), per_column(seen, state)


def attention(state, pos, seen):
    """Softmax over the seen positions times their values; a row that sees
    nothing gives 0 and -inf."""
    case = state["case"]
    N, R, Hkv, D = case["N"], case["R"], case["Hkv"], case["D"]
    score = torch.where(per_column(seen, state), products(state, pos), -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, tokens(state, pos, 1).contiguous()) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total)).squeeze(-1)
    out = out.view(N, Hkv, R, -1, D).transpose(1, 2).reshape(N * R, -1, D)
    return {"out": out.to(state["q"].dtype), "lse": lse.view(N, Hkv, R, -1).transpose(1, 2).reshape(N * R, -1)}


def plain_window(state):
    case = state["case"]
    W, sinks, R = case["window"], case["sinks"], case["R"]
    # the sinks, then what the rows' windows span
    span = state["lens"].long()[:, None] - (W + R - 1) + torch.arange(W + R - 1, device=DEVICE)
    pos = torch.cat((torch.arange(sinks, device=DEVICE).expand(case["N"], -1),
                     torch.where(span >= sinks, span, -1)), 1)
    s, e = state["starts"].view(-1, R, 1), state["ends"].view(-1, R, 1)
    at = pos[:, None]
    seen = (at >= s) & (at < e) & ((at < s + sinks) | (at >= e - W))
    return attention(state, pos.clamp(min=0), seen)


def plain_tree(state):
    case, mask = state["case"], state["mask"].long()
    pos = torch.arange(state["table"].shape[1] * case["P"], device=DEVICE)
    draft = pos - state["ends"].long()[:, None]
    word = mask.gather(1, (draft // 32).clamp(0, mask.shape[1] - 1)) >> (draft % 32)
    drafted = (draft >= 0) & (draft < case["R"]) & (word % 2 != 0)
    seen = (pos >= state["starts"][:, None]) & (draft < 0) | drafted
    return attention(state, pos.expand(case["N"], -1), seen)


def plain_weigh(state):
    case = state["case"]
    N, R, Hkv = case["N"], case["R"], case["Hkv"]
    score, seen = scores(state)
    lse = state["lse"].view(N, R, Hkv, -1).transpose(1, 2).reshape(N, Hkv, -1, 1)
    p = torch.exp(torch.where(seen & (lse > -math.inf), score - lse, -math.inf))
    state["weights"] += p.sum(2).sum(1)
    return {"weights": state["weights"]}


def plain_evict(state):
    case, w, keep = state["case"], state["weights"], state["case"]["keep"]
    n = state["lens"].long()[:, None]
    pos = torch.arange(w.shape[1], device=DEVICE).expand_as(w)
    rank = torch.where((pos < case["sinks"]) | (pos >= n - case["recent"]), math.inf, w)
    rank = torch.where(pos < n, rank, -math.inf)
    best = rank.sort(dim=1, descending=True, stable=True).indices[:, :keep]
    best = torch.nn.functional.pad(best, (0, keep - best.shape[1]), value=w.shape[1])
    best = torch.where(best < n, best, w.shape[1]).sort(1).values
    count = torch.minimum(n[:, 0], torch.full_like(n[:, 0], keep))
    real = torch.arange(keep, device=DEVICE) < count[:, None]
    state["kept"].zero_()
    some = min(keep, w.shape[1])
    state["kept"][:, :some] = torch.where(real, w.gather(1, torch.where(real, best, 0)), 0.0)[:, :some]
    k, v = moved(state, best, count, torch.zeros_like(count), keep)
    return {"listed": torch.where(real, best, -1).int(), "count": count.int(), "kept": state["kept"],
            "k": k, "v": v}


def plain_accept(state):
    k, v = moved(state, state["path"].long(), state["count"].long(), state["lens"].long(),
                 state["case"]["R"] + state["case"]["B"] - 1)
    return {"k": k, "v": v}


def moved(state, listed, count, first, width):
    """Moves the first count listed tokens of every request to its positions
    from first on, under new scales; returns what then stands from the first
    one's block on, `width` tokens of each request."""
    case, cache, table = state["case"], state["cache"], state["table"].long()
    N, Hkv, D, P, B = case["N"], case["Hkv"], case["D"], case["P"], case["B"]
    kind, most, dtype = case["codes"], listed.shape[1], TYPES[case["type"]]
    begin = first // B * B
    blocks = (most - 1) // B + 2  # blocks that a request's moved tokens can fall into
    pos = begin[:, None] + torch.arange(blocks * B, device=DEVICE)
    t = pos - first[:, None]
    old, new = t < 0, (t >= 0) & (t < count[:, None])
    live = old | new
    source = torch.where(new, listed.gather(1, t.clamp(0, most - 1)), torch.where(old, pos, 0))
    value = torch.stack((tokens(state, source, 0), tokens(state, source, 1)), 3)
    value = value.permute(0, 2, 1, 3, 4)  # [N, T, Hkv, 2, D]
    value = torch.where(live[:, :, None, None, None], value, 0.0)
    amax = torch.where(new[:, :, None, None], value.abs().amax(-1), 0.0)
    scale = power_of_two_scale(amax.view(N, blocks, B, Hkv, 2).amax(2), kind)
    n = 2 * Hkv * P * D
    page = table.gather(1, (pos // P).clamp(max=table.shape[1] - 1)).clamp(min=0)
    slot = pos % P
    codes_pool = cache[:, :n].view(-1, 2, Hkv, P, D)
    scale_pool = cache[:, n:n + 2 * Hkv * (P // B) * 4].view(torch.float32).view(-1, 2, Hkv, P // B)
    was = scale_pool[page[:, ::B], :, :, slot[:, ::B] // B].transpose(2, 3)
    keeps = old.view(N, blocks, B).any(2)[..., None, None]
    scale = torch.where(keeps, torch.maximum(scale, was), scale).repeat_interleave(B, 1)
    code = to_codes(value / scale[..., None], kind)
    n_, t_ = live.nonzero(as_tuple=True)
    codes_pool[page[n_, t_], :, :, slot[n_, t_]] = code[n_, t_].transpose(1, 2)
    scale_pool[page[n_, t_], :, :, slot[n_, t_] // B] = scale[n_, t_].transpose(1, 2)
    value = torch.where(live[:, :, None, None, None], from_codes(code, kind) * scale[..., None], 0.0)
    value = value[:, :width].to(dtype).reshape(N * width, Hkv, 2, D)
    return value[:, :, 0].contiguous(), value[:, :, 1].contiguous()


# ------------------------------------------------------- the work, and 64 bits

def work(case):
    """Inputs read once and outputs written once; of the cache, each position
    that some row sees (keys alone where nothing reads the values)."""
    if case["op"] == "rotate":
        heads = case["rows"] * (case["Hq"] + case["Hkv"])
        return {"bytes": 4 * heads * case["D"] + 4 * case["rows"] + 2 * case["rot"] + 4 * case["D"],
                "flops": 10 * heads * case["D"]}
    N, R, Hkv, D, B = case["N"], case["R"], case["Hkv"], case["D"], case["B"]
    lens = lengths(case)
    token = 2 * Hkv * (D + 4 / B)
    if case["op"] == "evict":
        kept = sum(min(n, case["keep"]) for n in lens)
        stride = -(-max(lens) // case["P"]) * case["P"]
        lists = 4 * sum(lens) + 4 * N * (case["keep"] + stride + 2)
        return {"bytes": lists + 3 * kept * token + N * case["keep"] * 2 * Hkv * D * 2, "flops": 0}
    if case["op"] == "accept":
        moved_tokens = sum(accepted(case))
        back = moved_tokens + sum(n % B for n in lens)
        wide = N * (R + B - 1) * 2 * Hkv * D * 2
        return {"bytes": (2 * moved_tokens + back) * token + wide + 4 * N * R, "flops": 0}
    rows = N * R
    head = 2 * 2 * rows * case["Hq"] * D + 4 * rows * (case["Hq"] + 2)
    if case["op"] == "tree":
        # about half of the drafts that stand before one are its ancestors at most
        seen = sum(n * R for n in lens) + N * R
        return {"bytes": head + 4 * rows * (-(-R // 32)) + (sum(lens) + N * R) * (token + 4 / case["P"]),
                "flops": 4 * D * case["Hq"] * seen}
    ends = ends_of(case)
    if case["op"] == "window":
        most = case["window"] + case["sinks"]
        seen = int(ends.clamp(max=most).sum())
        spans = [min(n, most + R - 1) for n in lens]
        return {"bytes": head + sum(spans) * (token + 4 / case["P"]), "flops": 4 * D * case["Hq"] * seen}
    positions = sum(lens)
    return {"bytes": head - 2 * rows * case["Hq"] * D + positions * (token / 2 + 4 / case["P"] + 8),
            "flops": 2 * D * case["Hq"] * int(ends.sum())}


def exact(case, seed):
    """The operators' definitions in 64 bits, a request and a head at a time."""
    s = prepare(case, seed)
    if case["op"] == "rotate":
        return exact_rotate(case, s)
    if case["op"] in ("evict", "accept"):
        return exact_move(case, s)
    N, R, Hq, Hkv, D = case["N"], case["R"], case["Hq"], case["Hkv"], case["D"]
    G, P = Hq // Hkv, case["P"]
    out = torch.zeros(N * R, Hq, D, dtype=torch.float64, device=DEVICE)
    lse = torch.full((N * R, Hq), -math.inf, dtype=torch.float64, device=DEVICE)
    weights = s["weights"].double() if case["op"] == "weigh" else None
    q64, table = s["q"].double(), s["table"].cpu()
    ends = s["ends"].long()
    for i in range(N):
        need = int((table[i] >= 0).sum())
        pages = s["cache"][table[i, :need].long().to(DEVICE)]
        rows = slice(i * R, (i + 1) * R)
        at = torch.arange(need * P, device=DEVICE)
        e = ends[rows, None]
        ok = at < e
        if case["op"] == "window":
            ok &= (at < case["sinks"]) | (at >= e - case["window"])
        if case["op"] == "tree":
            for x in range(R):
                bit = (s["mask"][rows, x // 32] >> (x % 32)) & 1
                ok |= (bit == 1)[:, None] & (at == e + x)
        used = ok.any(0).nonzero()[:, 0]  # what some row sees
        ok = ok[:, used]
        for h in range(Hkv):
            k = head_values(case, pages, 0, h)[used]
            v = head_values(case, pages, 1, h)[used]
            z = (q64[rows, h * G:(h + 1) * G].reshape(-1, D) @ k.T).view(R, G, -1) / math.sqrt(D)
            z.masked_fill_(~ok[:, None], -math.inf)
            if weights is not None:
                x = s["lse"][rows, h * G:(h + 1) * G].double()[..., None]
                weights[i, used] += torch.exp(z - torch.where(x == -math.inf, math.inf, x)).sum((0, 1))
                continue
            lse[rows, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
            p = torch.nan_to_num(torch.softmax(z, -1))
            out[rows, h * G:(h + 1) * G] = (p.view(R * G, -1) @ v).view(R, G, D)
    return {"out": out, "lse": lse} if weights is None else {"weights": weights}


def head_values(case, pages, w, h):
    """[positions, D] values of one head's keys (w = 0) or values (w = 1), in 64 bits."""
    Hkv, P, D, B = case["Hkv"], case["P"], case["D"], case["B"]
    a = (w * Hkv + h) * P * D
    b = 2 * Hkv * P * D + (w * Hkv + h) * (P // B) * 4
    c = grid_values(case["codes"]).to(DEVICE)[pages[:, a:a + P * D].long()].view(-1, P // B, B, D)
    x = pages[:, b:b + P // B * 4].contiguous().view(torch.float32).double()
    return (c * x[:, :, None, None]).view(-1, D)


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


def exact_rotate(case, s):
    rot, out = case["rot"], {}
    for name in ("q", "k"):
        x = s[name].double()
        norm = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
        y = x * s[name + "_weight"].double() / torch.sqrt(norm ** 2 / case["D"] + 1e-6)
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if case["pairs"] else (i, i + rot // 2)
            z = torch.complex(y[..., a], y[..., b])
            angle = s["positions"].double() * float(s["inv_freq"][i])
            z = z * torch.polar(torch.ones_like(angle), angle)[:, None]
            y[..., a], y[..., b] = z.real, z.imag
        out[name] = y
    return out


def exact_move(case, s):
    N, Hkv, D, P, B, kind = case["N"], case["Hkv"], case["D"], case["P"], case["B"], case["codes"]
    lens, evict = s["lens"].tolist(), case["op"] == "evict"
    width = case["keep"] if evict else case["R"] + B - 1
    out = torch.zeros(2, N, width, Hkv, D, dtype=torch.float64, device=DEVICE)
    kept = torch.zeros(s["weights"].shape, dtype=torch.float64, device=DEVICE) if evict else None
    table = s["table"].cpu()
    lists, counts = [], []
    for i in range(N):
        if evict:
            w, n = s["weights"][i, :lens[i]].double(), lens[i]
            must = torch.zeros(n, dtype=torch.bool, device=DEVICE)
            must[:case["sinks"]] = True
            must[max(0, n - case["recent"]):] = True
            rest = (~must).nonzero()[:, 0]
            free = max(0, min(n, case["keep"]) - int(must.sum()))
            must[rest[torch.sort(-w[rest], stable=True).indices[:free]]] = True
            chosen = must.nonzero()[:, 0]
            kept[i, :len(chosen)] = w[chosen]
            lists.append(torch.nn.functional.pad(chosen, (0, width - len(chosen)), value=-1))
            counts.append(len(chosen))
            first = 0
        else:
            first = lens[i]
            chosen = s["path"][i, :int(s["count"][i])].long()
        begin = first // B * B
        old, total = first - begin, first - begin + len(chosen)
        need = int((table[i] >= 0).sum())
        pages = s["cache"][table[i, :need].long().to(DEVICE)]
        source = torch.cat((torch.arange(begin, first, device=DEVICE), chosen))
        for w in (0, 1):
            for h in range(Hkv):
                z = torch.zeros(-(-total // B) * B, D, dtype=torch.float64, device=DEVICE)
                z[:total] = head_values(case, pages, w, h)[source]
                amax = z.abs().amax(1)
                amax[:old] = 0
                scale = amax.view(-1, B).amax(1) / (448.0 if kind == "e4m3" else 127.0)
                scale = torch.exp2(torch.ceil(torch.log2(scale.clamp(min=2.0 ** -126))))
                if old:
                    at = 2 * Hkv * P * D + ((w * Hkv + h) * (P // B) + begin % P // B) * 4
                    was = pages[begin // P, at:at + 4].clone().view(torch.float32)
                    scale[0] = torch.maximum(scale[0], was.double()[0])
                scale = scale.repeat_interleave(B)[:, None]
                out[w, i, :total, h] = (nearest(z / scale, kind) * scale)[:total]
    out = out.view(2, N * width, Hkv, D)
    more = {"listed": None, "count": None, "kept": kept} if evict else {}
    return {**more, "k": out[0], "v": out[1]}
