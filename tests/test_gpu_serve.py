"""GPU parity of the page plan and of the cache append against their
definitions (serve_ref.py): integers equal, copies bit for bit, rotations
within the bound of one bf16 rounding and a handful of fp32 ones."""
import numpy as np
import pytest

import serve_ref as ref

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


# ------------------------------------------------------------------ page plan

def plan_inputs(rng, B, max_pages, ps, slack, old, new):
    cap = max_pages * ps
    old, new = np.asarray(old, np.int32), np.asarray(new, np.int32)
    held = -(-np.clip(old, 0, cap) // ps)
    want = -(-np.clip(new, 0, cap) // ps)
    num = max(1, int(held.sum()) + int(np.maximum(want - held, 0).sum()) + slack)
    num = max(num, int(held.sum()))
    ids = rng.permutation(num).astype(np.int32)
    table = np.full((B, max_pages), -7, np.int32)
    k = 0
    for b in range(B):
        table[b, :held[b]] = ids[k:k + held[b]]
        k += held[b]
    head = int(rng.integers(0, num))
    ring = np.full(num, -5, np.int32)
    free = ids[k:]
    ring[(head + np.arange(len(free))) % num] = free
    return old, new, table, ring, np.array([head, len(free)], np.int32)


def check_plan(torch, eb, x, ps, N, index=None, bad=False):
    old, new, table, ring, state = x
    r = ref.plan(old, new, table, ring, state, ps, N, index)
    assert r[4] == bad
    d = [i32(torch, a) for a in x]
    ix = None if index is None else i32(torch, index)
    for _ in range(2):     # the same step again gives the same answer
        slots, out = eb.paged_plan(*d, ps, N, index=ix)
        assert eb.device_status() == (7 if bad else 0)
        for a, b, n in zip((slots, out, d[2], d[3]), r, ("slots", "state", "table", "ring")):
            assert np.array_equal(a.cpu().numpy(), b), n
    assert np.array_equal(d[4].cpu().numpy(), state)


PLANS = [
    # B, N, ps, max_pages, lo, hi, grow
    (1, 1, 1, 1, 0, 0, 1),
    (1, 1, 16, 4, 15, 16, 1),
    (5, 3, 8, 9, 0, 60, 3),
    (33, 31, 16, 20, 0, 250, 31),        # several sequences per CTA, an odd number of them
    (64, 16, 16, 40, 0, 500, 16),
    (257, 1, 16, 40, 0, 600, 1),         # more than a CTA's 64 sequences
    (2, 1024, 32, 70, 0, 900, 1024),     # one chunk exactly
    (3, 1025, 128, 20, 0, 1000, 1025),   # a chunk of one
    (2, 5000, 7, 900, 0, 1000, 5000),    # page sizes are any number here
    (2000, 2, 64, 12, 0, 700, 2),
]


@pytest.mark.parametrize("case", PLANS, ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("mode", ["grow", "mixed"])
def test_plan(torch, eb, case, mode):
    B, N, ps, mp, lo, hi, grow = case
    rng = np.random.default_rng(B * 131 + N)
    old = rng.integers(lo, hi + 1, B)
    new = old + rng.integers(0, grow + 1, B)
    if mode == "mixed":      # some finish, some roll back, some stay
        new = np.where(rng.random(B) < 0.3, 0, new)
        new = np.where(rng.random(B) < 0.2, old // 2, new)
    x = plan_inputs(rng, B, mp, ps, 3, old, new)
    check_plan(torch, eb, x, ps, N)


def test_plan_of_nodes_and_padding(torch, eb):
    """index: rejected nodes, places beyond the accepted length, the lowest
    and the largest int, the same place twice."""
    rng = np.random.default_rng(3)
    B, N, ps, mp = 6, 40, 16, 12
    old = np.array([0, 7, 16, 100, 150, 33])
    new = old + np.array([0, 5, 16, 40, 1, 3])
    index = rng.integers(-1, 20, (B, N)).astype(np.int32)
    index[0, :4] = [0, -2 ** 31, 2 ** 31 - 1, 5]
    check_plan(torch, eb, plan_inputs(rng, B, mp, ps, 0, old, new), ps, N, index)


def test_plan_lengths_are_clamped(torch, eb):
    rng = np.random.default_rng(4)
    x = plan_inputs(rng, 4, 3, 16, 2, [-5, 10, 48, 0], [20, 1000, -3, -(2 ** 31)])
    check_plan(torch, eb, x, 16, 50)


def test_plan_shortage_and_overflow_are_reported(torch, eb):
    rng = np.random.default_rng(5)
    old, new, table, ring, state = plan_inputs(rng, 5, 8, 16, 0, [16] * 5, [60, 17, 16, 90, 33])
    short = state.copy()
    short[1] = 4                     # pages for the first two requests and one of the next
    check_plan(torch, eb, (old, new, table, ring, short), 16, 80, bad=True)
    empty = np.array([state[0], 0], np.int32)
    check_plan(torch, eb, (old, new, table, ring, empty), 16, 80, bad=True)
    # a count that leaves no room for what is given back; a head outside the ring
    full = np.array([-3, len(ring)], np.int32)
    check_plan(torch, eb, (old, np.zeros(5, np.int32), table, ring, full), 16, 1, bad=True)
    # a table entry that cannot be one: its tokens get no slot
    t2 = table.copy()
    t2[1, 0] = 10 ** 6
    o2 = np.array([8, 8, 8, 8, 8], np.int32)
    check_plan(torch, eb, (o2, o2 + 4, t2, ring, state), 16, 8, bad=True)


def test_plan_leaves_other_entries_and_streams_alone(torch, eb):
    """On another stream than the tensors' own, into buffers of the caller."""
    rng = np.random.default_rng(6)
    x = plan_inputs(rng, 9, 20, 16, 4, rng.integers(0, 200, 9), rng.integers(0, 300, 9))
    r = ref.plan(*x, 16, 100)
    d = [i32(torch, a) for a in x]
    slots = torch.full((9, 100), 99, dtype=torch.int32, device="cuda")
    out = torch.zeros(2, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a, b = eb.paged_plan(*d, 16, 100, slots=slots, state_out=out, stream=s)
    s.synchronize()
    assert a is slots and b is out
    for got, want in zip((slots, out, d[2], d[3]), r):
        assert np.array_equal(got.cpu().numpy(), want)


# ------------------------------------------------------------------ append

def bf16(torch, rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32)).bfloat16().cuda()


def bits(t):
    import torch
    return t.contiguous().view(torch.int16).cpu()


APPENDS = [
    # B, N, Hq, Hkv, d, ps, pairing, fused, rope, keep
    (1, 1, 1, 1, 64, 8, 0, False, True, 1.0),
    (3, 1, 8, 2, 128, 16, 0, True, True, 1.0),
    (64, 1, 32, 8, 128, 16, 1, True, True, 1.0),
    (5, 7, 4, 4, 64, 32, 1, True, True, 0.6),
    (2, 63, 8, 1, 128, 16, 0, False, True, 0.1),
    (2, 700, 4, 2, 128, 64, 0, True, True, 1.0),     # tiles of 32 tokens, the last one ragged
    (3, 500, 2, 2, 64, 16, 1, False, True, 0.5),
    (4, 63, 0, 8, 128, 16, 0, False, False, 0.06),   # the accepted few, not rotated
    (1, 1, 0, 1, 64, 8, 0, True, False, 1.0),
    (3, 1100, 0, 2, 64, 100, 0, True, False, 0.0),   # nothing is stored; a contiguous cache's rows
]


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: "x".join(map(str, c)))
def test_append(torch, eb, case):
    B, N, Hq, Hkv, d, ps, pairing, fused, rope, keep = case
    rng = np.random.default_rng(N * 7 + d)
    if fused:
        x = bf16(torch, rng, B, N, Hq + 2 * Hkv, d).transpose(1, 2)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    else:
        q, k, v = (bf16(torch, rng, B, h, N, d) for h in (Hq, Hkv, Hkv))
    pages = -(-B * N // ps) + 3
    kc, vc = bf16(torch, rng, pages, Hkv, ps, d), bf16(torch, rng, pages, Hkv, ps, d)
    slots = rng.permutation(pages * ps)[:B * N].reshape(B, N).astype(np.int32)
    slots[rng.random((B, N)) >= keep] = -1 - rng.integers(0, 5)
    pos = rng.integers(0, 200000, (B, N)).astype(np.int32)
    want_k, want_v = kc.cpu().double(), vc.cpu().double()
    k64, v64 = k.cpu().double(), v.cpu().double()
    bound = torch.zeros_like(want_k)
    q64 = None
    if rope:
        kr = ref.rotate(k64, pos, 10000.0, pairing)
        kb = ref.rotate_bound(k64, kr, pairing)
        q64 = ref.rotate(q.cpu().double(), pos, 10000.0, pairing)
    else:
        kr, kb = k64, torch.zeros_like(k64)
    for b in range(B):
        for t in range(N):
            s = int(slots[b, t])
            if s >= 0:
                want_k[s // ps, :, s % ps] = kr[b, :, t]
                bound[s // ps, :, s % ps] = kb[b, :, t]
                want_v[s // ps, :, s % ps] = v64[b, :, t]
    qo, ko = eb.kv_append(k, v, i32(torch, slots), kc, vc, q=q if Hq else None,
                          positions=i32(torch, pos) if rope else None, rope_pairing=pairing,
                          return_k=rope)
    assert eb.device_status() == 0
    assert bool(((kc.cpu().double() - want_k).abs() <= bound).all())
    assert torch.equal(vc.cpu().double(), want_v)
    if rope:
        assert bool(((ko.cpu().double() - kr).abs() <= kb).all())
        qb = ref.rotate_bound(q.cpu().double(), q64, pairing)
        assert bool(((qo.cpu().double() - q64).abs() <= qb).all())
    else:
        assert qo is None and ko is None


@pytest.mark.parametrize("d,pairing,N", [(64, 0, 40), (128, 1, 40), (128, 0, 1500), (64, 1, 1500)])
def test_append_rotates_as_rope_apply(torch, eb, d, pairing, N):
    """At consecutive positions: the same bits, also in place."""
    rng = np.random.default_rng(d + N)
    q, k = bf16(torch, rng, 2, 4, N, d), bf16(torch, rng, 2, 2, N, d)
    pos = i32(torch, 1234 + np.tile(np.arange(N), (2, 1)))
    qr = eb.rope_apply(q, pos_offset=1234, pairing=pairing)
    kr = eb.rope_apply(k, pos_offset=1234, pairing=pairing)
    qo, ko = eb.kv_append(k, q=q, positions=pos, rope_pairing=pairing)
    assert torch.equal(bits(qo), bits(qr)) and torch.equal(bits(ko), bits(kr))
    qo, ko = eb.kv_append(k, q=q, positions=pos, rope_pairing=pairing, q_out=q, k_out=k)
    assert qo is q and ko is k
    assert torch.equal(bits(q), bits(qr)) and torch.equal(bits(k), bits(kr))


def test_append_specials_and_far_slots(torch, eb):
    """NaN and infinities are copied as they are, into the rows of their slot
    alone; a slot beyond the cache is reported and not stored."""
    rng = np.random.default_rng(9)
    k, v = bf16(torch, rng, 2, 2, 3, 64), bf16(torch, rng, 2, 2, 3, 64)
    k[0, 0, 0] = float("nan")
    v[1, 1, 2] = float("inf")
    kc = torch.zeros(4, 2, 8, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    slots = np.array([[31, 0, 2 ** 31 - 1], [32, -1, 5]], np.int32)
    assert eb.kv_append(k, v, i32(torch, slots), kc, vc) == (None, None)
    assert eb.device_status() == 7
    assert eb.device_status() == 0
    wk, wv = torch.zeros_like(kc), torch.zeros_like(vc)
    for b, t, s in [(0, 0, 31), (0, 1, 0), (1, 2, 5)]:
        wk[s // 8, :, s % 8], wv[s // 8, :, s % 8] = k[b, :, t], v[b, :, t]
    assert torch.equal(bits(kc), bits(wk)) and torch.equal(bits(vc), bits(wv))


def test_append_broadcast_and_single_sized_views(torch, eb):
    """A key head expanded over the heads (stride 0), and a stride over one
    token that no address uses."""
    rng = np.random.default_rng(10)
    k = bf16(torch, rng, 3, 1, 1, 128).expand(3, 4, 1, 128)
    v = bf16(torch, rng, 3, 4, 5, 128)[:, :, 2:3]
    kc = torch.zeros(3, 4, 2, 128, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    eb.kv_append(k, v, i32(torch, [[0], [3], [4]]), kc, vc)
    for b, s in enumerate([0, 3, 4]):
        assert torch.equal(kc[s // 2, :, s % 2], k[b, :, 0])
        assert torch.equal(vc[s // 2, :, s % 2], v[b, :, 0])


def test_append_rows_past_4_gib(torch, eb):
    """Byte offsets beyond 32 bits on the cache's side (5 GiB of keys)."""
    Hkv, ps, d = 8, 128, 128
    pages = 20480                     # 20480 * 8 * 128 rows of 256 bytes = 5 GiB
    kc = torch.zeros(pages, Hkv, ps, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    rng = np.random.default_rng(11)
    k, v = bf16(torch, rng, 1, Hkv, 3, d), bf16(torch, rng, 1, Hkv, 3, d)
    s = [pages * ps - 1, (pages - 1) * ps, 17000 * ps + 5]
    eb.kv_append(k, v, i32(torch, [s]), kc, vc)
    for t, x in enumerate(s):
        assert torch.equal(kc[x // ps, :, x % ps], k[0, :, t])
        assert torch.equal(vc[x // ps, :, x % ps], v[0, :, t])
    assert int((kc != 0).any(-1).sum()) == 3 * Hkv


# ------------------------------------------------------------------ together

def test_plan_and_append_in_a_graph_with_decode(torch, eb):
    """A decode step captured once and replayed: plan, append, paged decode.
    The replays equal the steps made one by one."""
    rng = np.random.default_rng(12)
    B, Hq, Hkv, d, ps, mp, steps = 3, 8, 2, 128, 16, 6, 20
    pages = 14
    lens0 = np.array([15, 0, 31], np.int32)
    xs = [bf16(torch, rng, B, 1, Hq + 2 * Hkv, d).transpose(1, 2) for _ in range(steps)]

    def fresh():
        s = dict(lens=i32(torch, np.zeros(B)), table=i32(torch, np.full((B, mp), -1)),
                 ring=i32(torch, np.arange(pages)), state=i32(torch, [0, pages]),
                 kc=torch.zeros(pages, Hkv, ps, d, dtype=torch.bfloat16, device="cuda"))
        s["vc"] = torch.zeros_like(s["kc"])
        lens = i32(torch, lens0)
        pre = bf16(torch, np.random.default_rng(1), B, 2 * Hkv, 31, d)
        slots, state = eb.paged_plan(s["lens"], lens, s["table"], s["ring"], s["state"], ps, 31)
        eb.kv_append(pre[:, :Hkv].contiguous(), pre[:, Hkv:].contiguous(), slots, s["kc"], s["vc"])
        s["lens"].copy_(lens)
        s["state"].copy_(state)
        s["x"] = torch.empty_like(xs[0])
        return s

    def step(s):
        new = s["lens"] + 1
        slots, state = eb.paged_plan(s["lens"], new, s["table"], s["ring"], s["state"], ps, 1)
        x = s["x"]
        q, _ = eb.kv_append(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], slots, s["kc"], s["vc"], q=x[:, :Hq],
                            positions=s["lens"][:, None].contiguous())
        o = eb.attn_fwd_paged(q, s["kc"], s["vc"], s["table"], new, return_lse=False)
        s["lens"].copy_(new)
        s["state"].copy_(state)
        return o

    a, outs = fresh(), []
    for x in xs:
        a["x"].copy_(x)
        outs.append(step(a).clone())
    g = fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):      # warm-up on copies of the state
        step({k: t.clone() for k, t in g.items()})
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step(g)
    for x, want in zip(xs, outs):
        g["x"].copy_(x)
        graph.replay()
        assert torch.equal(bits(o), bits(want))
    for n in ("lens", "table", "ring", "state", "kc", "vc"):
        assert torch.equal(a[n], g[n]), n
    assert eb.device_status() == 0
