"""Plain 64-bit implementation of the paged key/value cache's operators on the
CPU, and seeded caches for their tests. Nothing here uses the package."""
import math

import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # largest relative rounding


def code_values(codes):
    """What each of the 256 codes stands for."""
    c = np.arange(256)
    if codes == "int8":
        return torch.from_numpy((c - 256 * (c >= 128)).astype(np.float64))
    e, m = (c >> 3) & 15, c & 7
    a = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    a = np.where((c & 127) == 127, np.nan, a)
    return torch.from_numpy(np.where(c >= 128, -a, a))


def page_bytes(Hkv, D, P, B):
    return (2 * Hkv * (P * D + P // B * 4) + 127) // 128 * 128


class Pool:
    """Pages on the CPU: codes [pages, 2, Hkv, P, D] uint8, scales [pages, 2,
    Hkv, P / B] fp32, and the bytes they make."""

    def __init__(self, pages, Hkv, D, P, B, codes, seed, nan_codes=False):
        g = torch.Generator().manual_seed(seed)
        self.dims, self.kind = (Hkv, D, P, B), codes
        self.codes = torch.randint(0, 256, (pages, 2, Hkv, P, D), generator=g, dtype=torch.uint8)
        if codes == "e4m3" and not nan_codes:
            self.codes[(self.codes & 127) == 127] = 0x3A
        if codes == "e4m3":  # e4m3 bytes at random are mostly large: thin them out
            self.codes[..., ::2] &= 0xBF
        top = 448.0 if codes == "e4m3" else 127.0
        self.scales = torch.exp2(torch.randint(-3, 3, (pages, 2, Hkv, P // B), generator=g)) * 8 / top

    def bytes(self, gap=0):
        Hkv, D, P, B = self.dims
        n = 2 * Hkv * P * D
        out = torch.full((self.codes.shape[0], page_bytes(*self.dims) + gap), 0x5A, dtype=torch.uint8)
        out[:, :n] = self.codes.reshape(-1, n)
        m = 2 * Hkv * (P // B) * 4
        out[:, n:n + m] = self.scales.reshape(-1, m // 4).contiguous().view(torch.uint8)
        return out

    def tokens(self, table_row, positions):
        """Values (k, v), each [n, Hkv, D] float64, of a request's positions."""
        Hkv, D, P, B = self.dims
        page = torch.as_tensor(table_row).long()[positions // P].clamp(0, len(self.codes) - 1)
        slot = positions % P
        val = code_values(self.kind)
        return tuple(val[self.codes[page, w, :, slot].long()] *
                     self.scales[page, w, :, slot // B].double()[..., None] for w in (0, 1))


def attend(pool, q, table, starts, ends, scale=None, indices=None):
    """(out, lse, tol_out, tol_lse) in float64. The tolerances: the output's
    rounding; 2^-10 of sum p |v| for probabilities rounded to 11 bits and
    fp32 sums; and the fp32 dot products, off by at most D 2^-24 of
    sum_d |q_d k_d| (both kinds of error enter p relatively)."""
    Hkv, D, P, B = pool.dims
    rows, Hq, _ = q.shape
    R, G = rows // table.shape[0], Hq // Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    cap = min(table.shape[1] * P, 1 << 20)
    out = torch.zeros(rows, Hq, D, dtype=torch.float64)
    lse = torch.full((rows, Hq), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    memo = {}
    for r in range(rows):
        s = min(max(int(starts[r]), 0), cap)
        e = min(max(int(ends[r]), s), cap)
        if indices is None:
            pos = torch.arange(s, e)
        else:
            x = indices[r].long()
            pos = s + x[(x >= 0) & (x < e - s)]
        if not len(pos):
            continue
        if r // R not in memo:
            memo = {r // R: pool.tokens(table[r // R], torch.arange(cap))}
        k, v = (t[pos] for t in memo[r // R])
        x = q[r].double().view(Hkv, G, D)
        S = torch.einsum("hgd,nhd->hgn", x, k) * scale
        Sabs = torch.einsum("hgd,nhd->hgn", x.abs(), k.abs()).amax(-1) * scale
        p = torch.softmax(S, -1)
        out[r] = torch.einsum("hgn,nhd->hgd", p, v).reshape(Hq, D)
        lse[r] = torch.logsumexp(S, -1).reshape(Hq)
        absolute = torch.einsum("hgn,nhd->hgd", p, v.abs()).reshape(Hq, D)
        dot = (D * 2.0 ** -24 * Sabs).reshape(Hq)
        tol[r] = (2.0 ** -10 + 2 * dot)[:, None] * absolute
        tol_lse[r] = dot + 2.0 ** -20 * (1 + lse[r].abs())
    tol += U[q.dtype] * out.abs() + 2.0 ** -25
    return out, lse, tol, tol_lse


def differs(got, want, tol):
    """Where got is further from want than tol allows (NaN and infinities have
    to be alike): a count."""
    got = got.double().cpu()
    alike = (got == want) | (torch.isnan(got) & torch.isnan(want)) | ((got - want).abs() <= tol)
    return int((~alike).sum())


def nearest(x, codes):
    """x rounded to the values of codes, to nearest, ties to even."""
    if codes == "int8":
        return torch.round(x)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def append(pool, k, v, table, starts, counts=None):
    """The pool after storing: values only change through codes and scales, in
    float64."""
    Hkv, D, P, B = pool.dims
    N = table.shape[0]
    R = k.shape[0] // N
    val = code_values(pool.kind)
    top = 448.0 if pool.kind == "e4m3" else 127.0
    cap = min(table.shape[1] * P, 1 << 20)
    code_of = {float(x): i for i, x in reversed(list(enumerate(val.tolist()))) if x == x}
    for i in range(N):
        count = R if counts is None else min(max(int(counts[i]), 0), R)
        blocks = {}
        for t in range(count):
            pos = int(starts[i]) + t
            if 0 <= pos < cap and 0 <= int(table[i, pos // P]) < len(pool.codes):
                blocks.setdefault(pos // B, []).append((pos, i * R + t))
        for b, items in blocks.items():
            page, slot0 = int(table[i, b * B // P]), b * B % P
            kept = items[0][0] - b * B
            for w, x in ((0, k), (1, v)):
                new = torch.stack([x[row] for _, row in items]).double()  # [n, Hkv, D]
                for h in range(Hkv):
                    y = new[:, h]
                    finite = y[torch.isfinite(y)].abs()
                    amax = float(finite.max()) if finite.numel() else 0.0
                    e = -126
                    if amax > 0:
                        e = max(-126, math.frexp(amax / top)[1] - 2)
                        while amax > top * 2.0 ** e:
                            e += 1
                    scale, was = 2.0 ** e, float(pool.scales[page, w, h, slot0 // B])
                    if kept:
                        scale = max(scale, was)
                    old = val[pool.codes[page, w, h, slot0:slot0 + kept].long()] * was
                    z = torch.cat([old, y]) / scale
                    z = nearest(z.clamp(-top, top), pool.kind)
                    nan = torch.isnan(z)
                    c = torch.tensor([code_of[float(a)] if a == a else 0 for a in z.flatten().tolist()],
                                     dtype=torch.uint8).view(z.shape)
                    if pool.kind == "e4m3":
                        c[nan] = 0x7F
                        c[torch.signbit(z) & (z == 0)] = 0x80
                    if scale == was:  # kept codes are rounded again only where it grows
                        c[:kept] = pool.codes[page, w, h, slot0:slot0 + kept]
                    pool.codes[page, w, h, slot0:slot0 + kept + len(items)] = c
                    pool.scales[page, w, h, slot0 // B] = scale


def make_table(lens, P, seed, extra=1, spare=3):
    """Each length's pages from one random permutation; -1 past them."""
    need = [-(-max(n, 0) // P) for n in lens]
    perm = np.random.default_rng(seed).permutation(sum(need) + spare)
    table = torch.full((len(lens), max(need) + extra), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = torch.from_numpy(perm[at:at + n].astype(np.int32))
        at += n
    return table, sum(need) + spare
