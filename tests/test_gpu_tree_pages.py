"""Every page size at both head sizes, lengths about a tile's edges, in each
form of the kernel; and chains of more than 32 nodes in the narrow ones."""
import pytest

from test_gpu_tree import call, check, eb, make, torch, want  # noqa: F401

pytestmark = pytest.mark.gpu

HEADS = [(8, 2, 3), (6, 2, 15), (8, 1, 9), (16, 1, 20)]     # 12, 45, 72 and 320 rows a kv head


@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "x".join(map(str, h)))
@pytest.mark.parametrize("ps", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("full", [False, True], ids=["partial", "full"])
def test_page_sizes(torch, eb, d, ps, heads, full):  # noqa: F811
    Hq, Hkv, N = heads
    L = [1, 127, 128, 129, 0, 400]
    n = [N] * 6 if full else [N, 1, N - 1, 0, N, 2]
    x = make(torch, 6, Hq, Hkv, N, d, ps, L, n, seed=d + ps + Hq)
    o, lse = call(torch, eb, x)
    assert eb.device_status() == 0
    check(torch, o, lse, want(x))


@pytest.mark.parametrize("d,Hq,Hkv,N", [(64, 2, 2, 33), (128, 2, 2, 64), (64, 3, 3, 100), (128, 2, 1, 64),
                                        (128, 1, 1, 128)])
def test_long_chains_in_the_narrow_forms(torch, eb, d, Hq, Hkv, N):  # noqa: F811
    x = make(torch, 3, Hq, Hkv, N, d, 16, [70, 0, 300], [N, N - 1, 33], seed=N + d, kind="chain")
    o, lse = call(torch, eb, x)
    assert eb.device_status() == 0
    check(torch, o, lse, want(x))
