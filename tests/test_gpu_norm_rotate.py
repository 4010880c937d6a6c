"""Norm and rotation of query and key heads against the formulas in 64 bits: types,
layouts, both kinds of pairs, parts of a head, far positions, in place, strides."""
import math

import pytest
import torch

import fp8_mqa_logits_amd as mqa
from attend_ref import U
from gpu_helpers import say

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


def formula(x, weight, positions, inv_freq, eps, pairs):
    """(y, tolerance) in float64. The norm's sum of D squares and the products after it
    are fp32: (D / 2 + 6) 2^-24 of an element; sine and cosine are within 2^-20, with
    rounding in fp32 2^-19 of the pair; the result's own rounding."""
    D = x.shape[-1]
    y = x.double()
    if eps is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
        if weight is not None:
            y = y * weight.double()
    tol = (D / 2 + 6) * 2.0 ** -24 * y.abs()
    if inv_freq is not None:
        h = len(inv_freq)
        a = positions.double()[:, None, None] * inv_freq.double()
        at = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if pairs else (slice(0, h), slice(h, 2 * h))
        p, s = y[..., at[0]].clone(), y[..., at[1]].clone()
        y[..., at[0]] = p * torch.cos(a) - s * torch.sin(a)
        y[..., at[1]] = s * torch.cos(a) + p * torch.sin(a)
        both = ((D / 2 + 6) * 2.0 ** -24 + 2.0 ** -19) * (p.abs() + s.abs())
        tol[..., at[0]] = tol[..., at[1]] = both
    return y, tol + U[x.dtype] * (y.abs() + tol) + 2.0 ** -25


def check(got, x, *how):
    y, tol = formula(x.cpu(), *how)
    off = (got.double().cpu() - y).abs()
    assert got.dtype == x.dtype and got.shape == x.shape
    assert bool((off <= tol).all()), float((off / tol).max())


def inputs(rows, heads, kv_heads, D, dtype, seed=3, weight_type=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, heads + 2 * kv_heads, D, generator=g)
    x = (x * torch.exp2(torch.randn(rows, heads + 2 * kv_heads, 1, generator=g))).to(dtype)
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(weight_type or dtype) for _ in range(2)]
    return x, w[0], w[1]


def freqs(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2).double() / rot)).float()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("rows,heads,kv_heads,D,rot", [
    (1, 1, 0, 64, 64), (1, 32, 8, 128, 128), (3, 5, 1, 64, 16), (77, 28, 4, 128, 32),
    (130, 12, 12, 256, 256), (257, 40, 8, 64, 48), (511, 32, 8, 128, 128), (600, 33, 7, 128, 112),
    (19, 6, 2, 256, 240)])
def test_norm_and_rotation(rows, heads, kv_heads, D, rot, pairs, dtype):
    say(f"case: norm_rotate {rows} {heads} {kv_heads} {D} {rot} {pairs} {dtype}")
    x, qw, kw = inputs(rows, heads, kv_heads, D, dtype)
    x = x.cuda()
    q, k = x[:, :heads], x[:, heads:heads + kv_heads] if kv_heads else None
    g = torch.Generator().manual_seed(rows)
    pos = torch.randint(0, 1 << 20, (rows,), generator=g).int()
    f = freqs(rot)
    before = x.clone()
    got_q, got_k = mqa.mqa_norm_rotate(q, k, qw.cuda(), kw.cuda() if kv_heads else None, pos.cuda(),
                                       f.cuda(), pairs=pairs)
    torch.cuda.synchronize()
    assert torch.equal(x, before) and got_q.is_contiguous()
    check(got_q, q, qw, pos, f, 1e-6, pairs)
    if kv_heads:
        check(got_k, k, kw, pos, f, 1e-6, pairs)
    else:
        assert got_k is None


def test_parts_of_it():
    # no norm, no weights, no rotation, fp32 weights, another eps
    x, qw, kw = inputs(70, 8, 2, 128, BF16, weight_type=torch.float32)
    q, k = x[:, :8].cuda(), x[:, 8:10].cuda()
    pos, f = torch.arange(70).int(), freqs(64)
    a = (pos.cuda(), f.cuda())
    for weights, eps, turned in (((qw, kw), 1e-5, True), ((None, None), 0.5, True),
                                 ((qw, None), 1e-6, False), ((None, kw), 0.0, True),
                                 ((None, None), None, True)):
        w = [None if t is None else t.cuda() for t in weights]
        gq, gk = mqa.mqa_norm_rotate(q, k, *w, *(a if turned else (None, None)), eps=eps)
        how = (pos, f) if turned else (None, None)
        check(gq, q, weights[0], *how, eps, False)
        check(gk, k, weights[1], *how, eps, False)
    gq, gk = mqa.mqa_norm_rotate(q, k, None, None, None, None, eps=None)
    assert torch.equal(gq, q) and torch.equal(gk, k)


@pytest.mark.parametrize("rows", [5, 900])
def test_in_place_into_slices_and_other_strides(rows):
    x, qw, kw = inputs(rows, 8, 2, 128, FP16)
    pos, f = (torch.arange(rows) + 131000).int(), freqs(128, 500000.0)
    a = (qw.cuda(), kw.cuda(), pos.cuda(), f.cuda())
    whole = x.cuda()
    want = mqa.mqa_norm_rotate(whole[:, :8], whole[:, 8:10], *a)
    wide = torch.full((rows, 13, 160), 7.0, dtype=FP16, device="cuda")
    out = (wide[:, 1:9, 16:144], wide[:, 10:12, 16:144])
    mqa.mqa_norm_rotate(whole[:, :8], whole[:, 8:10], *a, q_out=out[0], k_out=out[1])
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    wide[:, 1:9, 16:144] = 7.0
    wide[:, 10:12, 16:144] = 7.0
    assert bool((wide == 7.0).all())
    values = whole[:, 10:].clone()
    got = mqa.mqa_norm_rotate(whole[:, :8], whole[:, 8:10], *a, q_out=whole[:, :8],
                              k_out=whole[:, 8:10])
    assert got[0].data_ptr() == whole.data_ptr()
    assert torch.equal(whole[:, :8], want[0]) and torch.equal(whole[:, 8:10], want[1])
    assert torch.equal(whole[:, 10:], values)
    # heads before rows in memory
    turned = x[:, :10].transpose(0, 1).contiguous().cuda().transpose(0, 1)
    got = mqa.mqa_norm_rotate(turned[:, :8], turned[:, 8:], *a)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rows_do_not_depend_on_the_others():
    # the same bits for a row alone and among many (both sizes of launches)
    x, qw, kw = inputs(700, 32, 8, 128, BF16)
    x, pos, f = x.cuda(), torch.arange(700).int().cuda(), freqs(128).cuda()
    a = (qw.cuda(), kw.cuda())
    many = mqa.mqa_norm_rotate(x[:, :32], x[:, 32:40], *a, pos, f)
    for r in (0, 1, 699):
        one = mqa.mqa_norm_rotate(x[r:r + 1, :32], x[r:r + 1, 32:40], *a, pos[r:r + 1], f)
        assert torch.equal(one[0], many[0][r:r + 1]) and torch.equal(one[1], many[1][r:r + 1])


def test_positions_of_any_size_and_sign():
    x, qw, _ = inputs(8, 2, 0, 64, FP16)
    pos = torch.tensor([0, 1, -1, -777777, 1 << 24, (1 << 24) + 1, 1 << 28, -(1 << 28)]).int()
    f = freqs(64, 1e6)
    q = x.cuda()
    got, _ = mqa.mqa_norm_rotate(q, None, qw.cuda(), None, pos.cuda(), f.cuda())
    check(got, q, qw, pos, f, 1e-6, False)


def test_zeros_infinities_and_nan_stay_in_their_head():
    x, qw, _ = inputs(4, 6, 0, 128, BF16)
    x[0, 0], x[1, 2, 5], x[2, 3, 100] = 0.0, math.nan, math.inf
    pos, f = torch.arange(4).int(), freqs(64)
    got, _ = mqa.mqa_norm_rotate(x.cuda(), None, qw.cuda(), None, pos.cuda(), f.cuda())
    got = got.cpu()
    assert bool((got[0, 0] == 0).all()) and bool(torch.isnan(got[1, 2]).all())
    # an infinity's head: x / inf = 0, and NaN where it stood (element 100 is not rotated)
    assert torch.isnan(got[2, 3]).nonzero()[:, 0].tolist() == [100]
    assert bool((got[2, 3, :100] == 0).all())
    fine = torch.ones(4, 6, dtype=torch.bool)
    fine[0, 0] = fine[1, 2] = fine[2, 3] = False
    y, tol = formula(x.nan_to_num(0.0, 0.0, 0.0), qw, pos, f, 1e-6, False)
    assert bool(((got.double() - y).abs() <= tol)[fine].all())


def test_another_stream_and_a_captured_call():
    x, qw, kw = inputs(33, 8, 2, 128, BF16)
    x, a = x.cuda(), (qw.cuda(), kw.cuda(), torch.arange(33).int().cuda(), freqs(128).cuda())
    want = mqa.mqa_norm_rotate(x[:, :8], x[:, 8:10], *a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mqa.mqa_norm_rotate(x[:, :8], x[:, 8:10], *a, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = torch.empty_like(want[0]), torch.empty_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mqa.mqa_norm_rotate(x[:, :8], x[:, 8:10], *a, q_out=out[0], k_out=out[1])
    for k in range(3):
        x.normal_()
        graph.replay()
        want = mqa.mqa_norm_rotate(x[:, :8], x[:, 8:10], *a)
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_refusals():
    x, qw, kw = inputs(4, 8, 2, 128, BF16)
    x, qw, kw = x.cuda(), qw.cuda(), kw.cuda()
    q, k, pos, f = x[:, :8], x[:, 8:10], torch.arange(4).int().cuda(), freqs(128).cuda()
    call = mqa.mqa_norm_rotate
    for bad in ((q.float(), k, qw, kw, pos, f), (q, k.half(), qw, kw, pos, f), (q, k, qw.half(), kw, pos, f),
                (q, k, qw.float(), kw, pos, f), (q, k, qw, kw, pos.long(), f), (q, k, qw, kw, pos, None),
                (q, k, qw, kw, None, f), (q, k, qw, kw, pos, f.double()), ([1], k, qw, kw, pos, f)):
        with pytest.raises(TypeError):
            call(*bad)
    for bad in ((q[0], k, qw, kw, pos, f), (q.cpu(), k, qw, kw, pos, f), (q, k[:3], qw, kw, pos, f),
                (q, k[..., :64], qw, kw, pos, f), (q, k, qw[:64], kw, pos, f), (q, k, qw, kw, pos[:3], f),
                (q[..., ::2], k[..., ::2], None, None, pos, f), (q, k, qw, kw, pos, f[:0])):
        with pytest.raises(ValueError):
            call(*bad)
    with pytest.raises(ValueError):
        call(q, k, qw, kw, pos, f, eps=None)
    with pytest.raises(ValueError):
        call(q, k, qw, kw, pos, f, q_out=torch.empty(4, 8, 64, dtype=BF16, device="cuda"))
    odd = torch.zeros(4, 10, 132, dtype=BF16, device="cuda")
    for bad in ((q, k, qw, kw, pos, freqs(24).cuda()), (q, k, qw, kw, pos, freqs(144).cuda()),
                (x[:, :8, :96], x[:, 8:10, :96], None, None, pos, freqs(32).cuda()),
                (odd[:, :8, :128], k, qw, kw, pos, f), (odd[:, :8, 4:], None, qw, None, pos, f)):
        with pytest.raises(mqa.MQAError):
            call(*bad)
    with pytest.raises(mqa.MQAError):
        call(q, k, qw, kw, pos, f, eps=-1.0)
    with pytest.raises(mqa.MQAError):
        call(q, k, qw, kw, pos, f, eps=math.nan)
    with pytest.raises(mqa.MQAError):  # one row of outputs for all
        call(q, k, qw, kw, pos, f, q_out=torch.empty(1, 8, 128, dtype=BF16, device="cuda").expand(4, -1, -1))
