"""paged_plan over many calls, shortages among them: what a request got in a
shortage comes back when it is finished or taken back, the entries that got no
page do not, so that every page stays in a table or in the queue, once."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    from exact_scaled_dot_fwd_b200 import build
    build.build()
    return t


@pytest.fixture(scope="module")
def eb(torch):
    import exact_scaled_dot_fwd_b200 as m
    return m


def i32(torch, x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def plan(old, new, table, ring, state, ps, N):
    """The definition, one request and one page at a time; free pages as a
    list.  Returns (slots, state, table, ring, whether ERANGE is recorded)."""
    table, ring = table.copy(), ring.copy()
    P, cap = len(ring), table.shape[1] * ps
    head, count = int(state[0]) % P, min(max(int(state[1]), 0), P)
    queue = [int(ring[(head + m) % P]) for m in range(count)]
    slots = np.full((len(old), N), -1, np.int32)
    taken, back, bad = 0, [], False
    for b in range(len(old)):
        o, n = (min(max(int(x), 0), cap) for x in (old[b], new[b]))
        have, want = -(-o // ps), -(-n // ps)
        for j in range(have, want):
            bad |= not queue
            table[b, j] = queue.pop(0) if queue else -1
            taken += bool(table[b, j] >= 0)
        back += [int(p) for p in table[b, want:have] if 0 <= p < P]
        for i in range(min(N, max(0, n - o))):
            page = int(table[b, (o + i) // ps])
            if 0 <= page < P:
                slots[b, i] = page * ps + (o + i) % ps
            else:
                bad = True
    bad |= len(back) > P - count
    back = back[:P - count]
    for m, p in enumerate(back):
        ring[(head + count + m) % P] = p
    return slots, np.array([(head + taken) % P, len(queue) + len(back)], np.int32), table, ring, bad


class Run:
    """Device and reference state side by side."""

    def __init__(self, torch, eb, B, mp, ps, pages, N, rng):
        self.torch, self.eb, self.ps, self.N, self.pages = torch, eb, ps, N, pages
        self.lens = np.zeros(B, np.int64)
        self.ref = [np.full((B, mp), -1, np.int32), rng.permutation(pages).astype(np.int32),
                    np.array([int(rng.integers(0, pages)), pages], np.int32)]
        self.dev = [i32(torch, x) for x in self.ref]

    def step(self, new):
        slots, state, table, ring, bad = plan(self.lens, new, *self.ref, self.ps, self.N)
        t, r, s = self.dev
        got, out = self.eb.paged_plan(i32(self.torch, self.lens), i32(self.torch, new), t, r, s,
                                      self.ps, self.N)
        assert self.eb.device_status() == (7 if bad else 0)
        for a, b, n in zip((got, out, t, r), (slots, state, table, ring),
                           ("slots", "state", "table", "ring")):
            assert np.array_equal(a.cpu().numpy(), b), n
        self.ref, self.dev, self.lens = [table, ring, state], [t, r, out], np.array(new)
        h, c = (int(x) for x in state)
        held = [int(p) for b, n in enumerate(self.lens) for p in table[b, :-(-int(n) // self.ps)]]
        free = [int(ring[(h + m) % self.pages]) for m in range(c)]
        assert sorted([p for p in held if p >= 0] + free) == list(range(self.pages))
        return bad


def test_a_dropped_request_gives_back_its_pages_alone(torch, eb):
    r = Run(torch, eb, 3, 8, 16, 4, 64, np.random.default_rng(0))
    assert r.step([16, 64, 16])          # four pages for six
    assert not r.step([16, 0, 16])       # the second request is dropped: three pages
    assert r.ref[2][1] == 3
    assert not r.step([16, 48, 0])       # (the third has none to give back)
    assert not r.step([0, 0, 0])
    assert r.ref[2][1] == 4


def test_taken_back_to_any_length(torch, eb):
    r = Run(torch, eb, 2, 10, 8, 5, 80, np.random.default_rng(1))
    assert r.step([24, 80])              # 3 pages, then 2 of 10
    assert not r.step([24, 70])          # only entries without a page
    assert not r.step([24, 12])
    assert not r.step([24, 5])           # a page, with the queue empty
    assert not r.step([32, 5])
    assert not r.step([0, 5])
    assert not r.step([0, 40])
    assert not r.step([0, 0])


@pytest.mark.parametrize("B,N,ps,mp,pages", [
    (1, 7, 4, 9, 5),
    (5, 33, 16, 40, 60),
    (70, 9, 8, 20, 400),           # several sequences a CTA
    (300, 1, 16, 70, 6000),        # five CTAs of 64 sequences
    (200, 300, 8, 300, 20000),     # 67 CTAs of 3
    (3, 1500, 2, 2000, 3000),      # two CTAs a sequence
    (9, 1024, 1, 3000, 9000),      # one sequence a CTA
])
def test_runs_with_shortages(torch, eb, B, N, ps, mp, pages):
    rng = np.random.default_rng(B + N)
    r = Run(torch, eb, B, mp, ps, pages, N, rng)
    fair = pages * ps // B             # tokens a request may have on average
    shortages = 0
    for it in range(14):
        new = np.minimum(r.lens + rng.integers(0, fair + 2, B), mp * ps)
        u = rng.random(B) if it > 3 else np.ones(B)   # (at first they only grow)
        new = np.where(u < 0.15, 0, new)                                    # finished
        new = np.where((u > 0.15) & (u < 0.35), r.lens * rng.random(B), new)    # taken back
        if it == 9:
            new = np.zeros(B)              # all of them at once
        shortages += r.step(new.astype(np.int64))
    assert shortages
    r.step(np.zeros(B, np.int64))
    assert r.ref[2][1] == pages


def test_entries_that_are_no_pages_are_passed_over(torch, eb):
    table = np.array([[0, 10 ** 6, 3, -2 ** 31, 2 ** 31 - 1, 7], [8, 1, 2, 9, 4, 5]], np.int32)
    ring = np.full(8, -1, np.int32)
    state = np.array([6, 0], np.int32)
    old, new = [48, 40], [0, 8]
    want = plan(old, new, table, ring, state, 8, 2)
    d = [i32(torch, x) for x in (old, new, table, ring, state)]
    slots, out = eb.paged_plan(*d, 8, 2)
    assert eb.device_status() == 0
    for a, b in zip((slots, out, d[2], d[3]), want):
        assert np.array_equal(a.cpu().numpy(), b)
    # (there is no page 8 or 9 in a pool of 8)
    assert out.tolist() == [6, 6]
    assert d[3].tolist() == [7, 1, 2, 4, -1, -1, 0, 3]
