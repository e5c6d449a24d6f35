"""Many whole units a CTA, every node live: the Q tiles come by TMA, into
buffers through which the segment before the last one added up its row copies.
Against the 64-bit reference, and the same bits on every call."""
import pytest

from test_gpu_tree import check, call, eb, make, torch, want  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [
    # B, Hq, Hkv, Nq, d, page size (0: contiguous), keys: 768 units or more
    (96, 8, 8, 1, 64, 16, 150),          # 1 row
    (96, 32, 8, 8, 128, 16, 130),        # 32 rows: four copies
    (96, 32, 8, 8, 64, 0, 260),
    (96, 32, 8, 9, 128, 64, 140),        # 36 rows: two copies
    (96, 64, 8, 8, 64, 8, 129),          # 64 rows
    (110, 56, 7, 8, 128, 128, 200),
    (96, 80, 8, 8, 128, 16, 140),        # 80 rows: one
], ids=lambda c: "x".join(map(str, c)))
def test_many_whole_units(torch, eb, case):  # noqa: F811
    *sizes, keys = case
    B, N = case[0], case[3]
    x = make(torch, *sizes, [keys - i % 7 for i in range(B)], [N] * B, seed=sum(case))
    first = call(torch, eb, x)
    assert eb.device_status() == 0
    check(torch, *first, want(x))
    for _ in range(5):
        again = call(torch, eb, x)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
