"""The serving calls on another stream than the current one: what they
allocate is not memory that work queued on the current stream still uses, nor
given away while the current stream reads it."""
import pytest

pytestmark = pytest.mark.gpu

BUSY = 100_000_000          # clock cycles: some 50 ms


@pytest.fixture(scope="module")
def torch():
    import torch as t
    from exact_scaled_dot_fwd_b200 import build
    build.build()
    return t


def calls(torch, name):
    """A function that makes the call's inputs and returns a function of a
    stream that makes the call and returns its tensors."""
    import exact_scaled_dot_fwd_b200 as eb
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    bf = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    B, Hq, Hkv, N, d, ps = 2, 32, 8, 64, 128, 16
    q, k, v = bf(B, Hq, N, d), bf(B, Hkv, N, d), bf(B, Hkv, N, d)
    pos = torch.arange(N, dtype=torch.int32, device="cuda").repeat(B, 1)
    parents = pos - 1
    cache, lens = bf(B, Hkv, 256, d), i32([200, 256])
    old, new, state = i32([0, 0]), i32([60, 33]), i32([0, 8])
    table, ring = i32([[-1] * 4] * 2), torch.arange(8, dtype=torch.int32, device="cuda")

    def plan():
        t, r = table.clone(), ring.clone()
        return lambda stream: eb.paged_plan(old, new, t, r, state, ps, 4096, stream=stream)

    return {
        "plan": plan,
        "append": lambda: lambda stream: eb.kv_append(k, q=q, positions=pos, stream=stream),
        "tree": lambda: lambda stream: eb.attn_fwd_tree(q, cache, cache, lens, k, v, parents,
                                                        stream=stream),
    }[name]


@pytest.mark.parametrize("name", ["plan", "append", "tree"])
def test_memory_that_the_current_stream_still_writes(torch, name):
    """The current stream is held up, and behind that writes a freed block of
    each output's size: the results must not be in it."""
    make = calls(torch, name)
    side = torch.cuda.Stream()
    want = make()(None)
    for _ in range(3):
        call = make()
        freed = [torch.empty_like(t) for t in want]
        freed.append(torch.empty(1 << 25, dtype=torch.uint8, device="cuda"))   # a workspace's
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        for t in freed:
            t.fill_(77)
        del freed, t
        got = call(side)
        side.synchronize()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["plan", "append", "tree"])
def test_results_that_the_current_stream_still_reads(torch, name):
    """Results freed while the current stream has yet to read them are not
    handed to the next call on the side stream."""
    call = calls(torch, name)()
    side = torch.cuda.Stream()
    want = call(None)
    torch.cuda.synchronize()
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    copies = [t.clone() for t in got]
    del got
    with torch.cuda.stream(side):       # what takes the same sizes there next
        for t in want:
            torch.empty_like(t).fill_(55)
    torch.cuda.synchronize()
    for a, b in zip(copies, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["append", "tree"])
def test_captured_on_a_forked_stream(torch, name):
    """A capture that forks to a side stream for the call and joins it again."""
    call = calls(torch, name)()
    side = torch.cuda.Stream()
    want = call(None)
    call(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = call(side)
        torch.cuda.current_stream().wait_stream(side)
        copies = [t.clone() for t in got]
    for _ in range(3):
        for t in (*got, *copies):
            t.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(got, copies, want):
            assert torch.equal(a, c) and torch.equal(b, c)
