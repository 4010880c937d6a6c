"""Plain 64-bit implementations, on the CPU, of what a serving step does around
attention over the paged 8-bit cache. Nothing here uses the package."""
import math

import torch

from attend_ref import U


def ranges(starts, ends, cap):
    """Rows' ranges as the contract clamps them, [rows, 1] each."""
    s = starts.long().clamp(0, cap)[:, None]
    return s, torch.maximum(ends.long().clamp(max=cap)[:, None], s)


def window_seen(starts, ends, window, sinks, cap):
    """[rows, cap] bool: the last `window` and the first `sinks` positions of each range."""
    s, e = ranges(starts, ends, cap)
    at = torch.arange(cap)
    return (at >= s) & (at < e) & ((at < s + sinks) | (at >= e - window))


def tree_seen(starts, ends, mask, cap):
    """[rows, cap] bool: each range and the drafts behind it that the row's bits name."""
    s, e = ranges(starts, ends, cap)
    at = torch.arange(cap)
    x = at - e
    word = mask.long().gather(1, (x // 32).clamp(0, mask.shape[1] - 1))
    drafts = (x >= 0) & (x < 32 * mask.shape[1]) & ((word >> (x % 32)) % 2 != 0)
    return (at >= s) & (at < e) | drafts


def words(bits):
    """[rows, n] bool -> [rows, ceil(n / 32)] int32."""
    bits = torch.nn.functional.pad(bits, (0, -bits.shape[1] % 32)).view(len(bits), -1, 32)
    w = (bits.long() << torch.arange(32)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).int()


def attend(pool, q, table, seen, scale=None):
    """(out, lse, tol_out, tol_lse) in float64, rows seeing what `seen` [rows, cap] says.
    The tolerances: the output's rounding; 2^-10 of sum p |v| for probabilities
    rounded to 11 bits and fp32 sums; and the fp32 dot products, off by at most D
    2^-24 of sum_d |q_d k_d| (both kinds of error enter p relatively). The
    logarithm of the sums is formed from fp32 exponents to base 2 between 16 and 32, for
    the scales and scores of these tests: log2 of a value scale (one last place, 2^-19),
    its sum with a constant and its difference from the reference point (half a last
    place each, 2^-20): ln 2 (2^-19 + 2 * 2^-20) < 2^-18 at any lse, and 2^-20 of lse for
    the rest (that mqa_attend_paged is off by 1.3e-6 at an lse of 0.01 was measured)."""
    Hkv, D, P, B = pool.dims
    rows, Hq, _ = q.shape
    N, cap = table.shape[0], seen.shape[1]
    R, G = rows // N, Hq // Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    out = torch.zeros(rows, Hq, D, dtype=torch.float64)
    lse = torch.full((rows, Hq), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for i in range(N):
        used = seen[i * R:(i + 1) * R].any(0).nonzero()[:, 0]
        if not len(used):
            continue
        k, v = (t.transpose(0, 1) for t in pool.tokens(table[i], used))  # [Hkv, n, D]
        step = max(1, (1 << 24) // (Hq * len(used)))
        for a in range(i * R, (i + 1) * R, step):
            b = min(a + step, (i + 1) * R)
            see = seen[a:b, used]
            x = q[a:b].double().view(b - a, Hkv, G, D).transpose(0, 1).reshape(Hkv, -1, D)
            col = see[:, None].expand(-1, G, -1).reshape(1, -1, len(used))
            S = torch.where(col, x @ k.transpose(1, 2) * scale, -math.inf)
            Sabs = (x.abs() @ k.abs().transpose(1, 2)).masked_fill(~col, 0).amax(-1) * scale
            top = S.amax(-1, keepdim=True)
            p = torch.where(col, torch.exp(S - torch.where(top == -math.inf, 0.0, top)), 0.0)
            total = p.sum(-1, keepdim=True)
            p = p / torch.where(total == 0, 1.0, total)

            def rows_of(t):
                return t.view(Hkv, b - a, G, -1).transpose(0, 1).reshape(b - a, Hq, -1)

            out[a:b] = rows_of(p @ torch.where(torch.isnan(v), 0.0, v))
            bad = (col.double().expand(Hkv, -1, -1) @ torch.isnan(v).double()) > 0
            out[a:b] = torch.where(rows_of(bad), math.nan, out[a:b])
            lse[a:b] = rows_of(torch.log(total) + top)[..., 0]
            dot = D * 2.0 ** -24 * rows_of(Sabs[..., None])
            tol[a:b] = (2.0 ** -10 + 2 * dot) * rows_of(p @ v.abs().nan_to_num(0.0))
            tol_lse[a:b] = dot[..., 0] + 2.0 ** -18 + 2.0 ** -20 * lse[a:b].abs()
    tol += U[q.dtype] * out.abs() + 2.0 ** -25
    return out, lse, tol, tol_lse
