"""GPU test of ns_moe_sort at the most slots it takes, against the closed form for experts in turn."""

import pytest

import newton_schulz_quintic_amd as nsq
from tests.helpers import log

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("slots", [2 ** 31 - 1, 2 ** 31 - 511])
def test_moe_sort_of_the_most_slots(slots):
    """Slot s chooses expert s % 5: its row is the expert's first one plus s // 5. 26 GB of maps."""
    import torch
    log(f"sort {slots}")
    experts, step = 5, 1 << 27
    ids = torch.empty(slots, dtype=torch.int32, device="cuda")
    for a in range(0, slots, step):
        z = min(a + step, slots)
        ids[a:z] = torch.arange(a, z, device="cuda") % experts
    off = torch.empty(experts + 1, dtype=torch.int32, device="cuda")
    slot = torch.full((slots,), -9, dtype=torch.int32, device="cuda")
    row = torch.full((slots, 1), -9, dtype=torch.int32, device="cuda")
    nsq.ns_moe_sort(ids.view(-1, 1), experts, off, slot, row)
    torch.cuda.synchronize()
    first = [0]
    for e in range(experts):
        first.append(first[-1] + (slots - e + experts - 1) // experts)
    assert off.tolist() == first
    starts = torch.tensor(first, device="cuda")
    for a in range(0, slots, step):
        z = min(a + step, slots)
        s = torch.arange(a, z, device="cuda")
        want = starts[s % experts] + s // experts
        assert torch.equal(row[a:z, 0].long(), want)
        assert torch.equal(slot[want].long(), s)
