"""Workspaces of attention calls: one that is sized for the largest batch serves
every smaller one, and a call that the binding sizes takes what it needs."""
import pytest
import torch

import attend_ref as ref
import fp8_mqa_logits_amd as mqa
from fp8_mqa_logits_amd import attend as A
from gpu_helpers import say
from test_gpu_attend import layout, lists, problem

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (64, 1, 128), (40, 8, 64), (12, 12, 64)])
@pytest.mark.parametrize("requests,R,positions", [(512, 1, 131072), (96, 7, 20000), (1, 4096, 49152),
                                                  (3, 700, 1 << 20), (1, 1, 777)])
def test_the_largest_batch_s_workspace_serves_smaller_ones(requests, R, positions, Hq, Hkv, D):
    L, lib = mqa.KVLayout(Hkv, D), A._load()
    most = mqa.workspace_size_attend(requests, R, Hq, L, positions)
    for n in sorted({1, 2, 5, 24, 31, 32, 64, 95, 300, 511, requests}):
        for r in sorted({1, 2, 4, 16, 33, 100, 333, 699, 2048, R}):
            for p in (64, 512, 777, 4096, 19999, 49151, 131072, positions):
                if n > requests or r > R or p > positions:
                    continue
                for listed in (0, 1):
                    need = lib.workspace_size_attend_call(n, r, Hq, Hkv, D, p, listed, 0)
                    assert 0 < need <= most, (n, r, p, listed)


def test_positions_past_the_largest_context():
    # a table's room may be larger than the positions that a request can have
    L = mqa.KVLayout(8, 128)
    size = A._load().workspace_size_attend
    assert size(4, 1, 32, 8, 128, (1 << 31) - 1, 0) == size(4, 1, 32, 8, 128, 1 << 20, 0)
    call = A._load().workspace_size_attend_call
    assert call(4, 1, 32, 8, 128, (1 << 31) - 1, 0, 0) == call(4, 1, 32, 8, 128, 1 << 20, 0, 0)
    assert mqa.workspace_size_attend(4, 1, 32, L, 1 << 20) > 256


@pytest.mark.parametrize("lens", [[900], [900, 41, 333]])
def test_calls_of_smaller_batches(lens):
    say(f"case: smaller batch {lens}")
    pool, table, q, starts, ends = problem(lens, 1, 32, 8, 128, 64, 64, BF16, "e4m3", extra=2048)
    L = layout(pool)
    work = torch.empty(mqa.workspace_size_attend(512, 4, 32, L, 131072 + 1024 * 64),
                       dtype=torch.uint8, device="cuda")
    args = (q.cuda(), pool.bytes().cuda(), table.cuda())
    want, _, tol, _ = ref.attend(pool, q, table[:, :15], starts, ends)
    out = mqa.mqa_attend_paged(L, *args, starts.cuda(), ends.cuda(), workspace=work)
    assert ref.differs(out, want, tol) == 0
    idx = lists(starts, ends, 2048, 3)
    want, _, tol, _ = ref.attend(pool, q, table[:, :15], starts, ends, indices=idx)
    out = mqa.mqa_attend_topk(L, *args, idx.cuda(), starts.cuda(), ends.cuda(), workspace=work)
    assert ref.differs(out, want, tol) == 0


def test_a_listed_call_takes_what_it_needs():
    # lists whose rows fill the card need no parts; a range of as many positions would
    lib = A._load()
    assert lib.workspace_size_attend_call(32, 4, 32, 8, 128, 2048, 1, 0) == 256
    assert lib.workspace_size_attend_call(1, 1, 32, 8, 128, 131072, 0, 0) > 256
