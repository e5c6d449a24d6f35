"""paged_plan on a table of 2^31 - 1 entries (8 GiB, and 8 GiB of free pages):
steps over a row must not pass its end in 32 bits."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [300000, 1500000])
def test_plan_of_the_longest_row(N):
    import torch
    from exact_scaled_dot_fwd_b200 import build
    import exact_scaled_dot_fwd_b200 as eb
    build.build()
    P = 2 ** 31 - 1
    i32 = dict(dtype=torch.int32, device="cuda")
    ring = torch.arange(P, **i32)
    table = torch.full((1, P), -1, **i32)
    old, new = torch.tensor([10], **i32), torch.tensor([P], **i32)
    table[0, :10] = torch.arange(10, **i32)
    state = torch.tensor([10, P - 10], **i32)          # pages 0 .. 9 are held
    slots, state = eb.paged_plan(old, new, table, ring, state, 1, N)
    assert eb.device_status() == 0
    assert state.tolist() == [0, 0]
    assert torch.equal(slots[0], torch.arange(10, 10 + N, **i32))
    assert bool((table[0] == ring).all())               # entry j is page j
    back = P - 4999
    slots, state = eb.paged_plan(new, torch.tensor([back], **i32), table, ring, state, 1, N)
    assert eb.device_status() == 0
    assert state.tolist() == [0, 4999] and bool((slots == -1).all())
    assert torch.equal(ring[:4999], table[0, back:])
