"""Selection for as many requests as a call may have."""
import pytest
import torch

import fp8_mqa_logits_amd as mqa
from gpu_helpers import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("requests,width", [(1 << 20, 40), ((1 << 16) - 1, 4097), (1 << 16, 4097),
                                            (840001, 4097), (1 << 20, 4500)])
def test_the_heaviest_of_many_requests(requests, width):
    # one weight of each request is the largest, the others are equal: the lowest position
    # besides it stays
    say(f"case: select {requests} x {width}")
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    at = torch.randint(0, width, (requests,), generator=g, device="cuda")
    w = torch.zeros(requests, width, device="cuda")
    w.scatter_(1, at[:, None], 1.0)
    length = torch.full((requests,), width, dtype=torch.int32, device="cuda")
    length[::1000] = 0
    length[1::1000] = 1
    kept = torch.full_like(w, 7.0) if width < 100 else None
    listed, count = mqa.mqa_kv_select(w, length, 3, kept=kept)
    del w
    # the two lowest positions besides the heaviest, and it, in ascending order
    low = torch.where(at == 0, 1, 0), torch.where(at <= 1, 2, 1)
    want = torch.stack((*low, at), 1).sort(1).values.int()
    want[::1000] = -1
    want[1::1000] = torch.tensor([0, -1, -1], dtype=torch.int32, device="cuda")
    assert torch.equal(listed, want)
    assert torch.equal(count, length.clamp(max=3))
    if kept is not None:
        heavy = (listed == at[:, None]) & (listed >= 0)
        assert torch.equal(kept[:, :3], heavy.float()) and not bool(kept[:, 3:].any())
