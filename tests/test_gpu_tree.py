"""GPU parity of attention for a tree of drafted tokens over a cache against
the 64-bit reference (serve_ref.tree), within its bounds.

Pages are shuffled; pages no sequence owns, cache rows past a sequence's
length and drafted rows past its nodes hold NaN, unused table entries are
-1."""
import math

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


def random_tree(rng, B, N, kind="random"):
    if kind == "chain":
        return np.tile(np.arange(-1, N - 1, dtype=np.int32), (B, 1))
    if kind == "roots":
        return np.full((B, N), -1, np.int32)
    return (np.floor(rng.random((B, N)) * (np.arange(N) + 1)) - 1).astype(np.int32)


def make(torch, B, Hq, Hkv, N, d, ps, L, n, seed, kind="random", qstd=2.0, cap=None):
    rng = np.random.default_rng(seed)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32)).bfloat16()
    L, n = np.asarray(L, np.int32), np.asarray(n, np.int32)
    x = dict(B=B, Hq=Hq, Hkv=Hkv, N=N, d=d, ps=ps, L=L, n=n, parents=random_tree(rng, B, N, kind),
             q=t(B, Hq, N, d) * qstd, kn=t(B, Hkv, N, d), vn=t(B, Hkv, N, d))
    x["k"] = [t(Hkv, max(1, int(l)), d) for l in L]
    x["v"] = [t(Hkv, max(1, int(l)), d) for l in L]
    nan = float("nan")
    for b in range(B):
        for s in ("q", "kn", "vn"):
            x[s][b, :, int(n[b]):] = nan
    if ps:
        held = -(-L // ps)
        mp = max(1, int(held.max())) + 1
        pages = int(held.sum()) + 2
        ids = rng.permutation(pages).astype(np.int32)
        x["table"] = np.full((B, mp), -1, np.int32)
        kc = torch.full((pages, Hkv, ps, d), nan, dtype=torch.bfloat16)
        vc = kc.clone()
        at = 0
        for b in range(B):
            for j in range(held[b]):
                p = int(ids[at])
                at += 1
                x["table"][b, j] = p
                m = min(ps, int(L[b]) - j * ps)
                kc[p, :, :m] = x["k"][b][:, j * ps:j * ps + m]
                vc[p, :, :m] = x["v"][b][:, j * ps:j * ps + m]
    else:
        cap = cap or max(1, int(L.max()))
        x["table"] = None
        kc = torch.full((B, Hkv, cap, d), nan, dtype=torch.bfloat16)
        vc = kc.clone()
        for b in range(B):
            kc[b, :, :L[b]], vc[b, :, :L[b]] = x["k"][b][:, :L[b]], x["v"][b][:, :L[b]]
    x["kc"], x["vc"] = kc, vc
    return x


def call(torch, eb, x, **kw):
    table = None if x["table"] is None else i32(torch, x["table"])
    return eb.attn_fwd_tree(x["q"].cuda(), x["kc"].cuda(), x["vc"].cuda(), i32(torch, x["L"]),
                            x["kn"].cuda(), x["vn"].cuda(), i32(torch, x["parents"]),
                            new_lens=i32(torch, x["n"]), block_table=table, **kw)


def want(x, scale=None):
    z = lambda t: t.double()
    return ref.tree(z(x["q"]), [z(k) for k in x["k"]], [z(v) for v in x["v"]], x["L"], z(x["kn"]),
                    z(x["vn"]), x["parents"], x["n"], scale or 1 / math.sqrt(x["d"]))


def check(torch, o, lse, w):
    ow, lw, to, tl = w
    o, lse = o.cpu().double(), lse.cpu().double()
    assert bool(torch.isfinite(o).all())
    assert bool(((o - ow).abs() <= to).all()), float(((o - ow).abs() - to).max())
    live = torch.isfinite(lw)
    assert torch.equal(torch.isfinite(lse), live) and not bool(torch.isnan(lse).any())
    assert bool(((lse - lw).abs()[live] <= tl[live]).all())
    assert bool((o[~live] == 0).all()) and bool((lse[~live] == -math.inf).all())


CASES = [
    # B, Hq, Hkv, Nq, d, page size (0: contiguous), cached lengths, nodes
    (1, 1, 1, 1, 64, 0, [1], [1]),
    (1, 1, 1, 1, 128, 8, [0], [1]),                                  # an empty cache
    (2, 4, 2, 3, 128, 16, [5, 0], [3, 0]),                           # a sequence without nodes
    (3, 8, 2, 5, 64, 16, [127, 128, 129], [5, 1, 4]),                # a tile's edges
    (3, 8, 2, 5, 128, 16, [127, 128, 129], [5, 1, 4]),
    (2, 6, 2, 21, 128, 32, [255, 700], [21, 20]),                    # 63 rows per kv head
    (2, 7, 1, 19, 64, 64, [1000, 3], [19, 11]),                      # 133 rows, one head odd
    (2, 8, 2, 32, 128, 128, [513, 130], [32, 31]),                   # 128 rows: one row tile
    (2, 4, 1, 33, 128, 8, [300, 90], [33, 7]),                       # 132 rows: a second one of 4
    (1, 8, 2, 64, 128, 16, [1029], [64]),                            # 256 rows
    (2, 16, 2, 33, 64, 8, [200, 777], [33, 30]),                     # 264 rows: two groups of tiles
    (1, 9, 1, 64, 128, 0, [333], [60]),                              # 576 rows
    (1, 2, 1, 128, 128, 16, [70], [128]),                            # one full tile of drafts
    (1, 2, 1, 129, 64, 16, [70], [129]),                             # a second tile of drafts
    (2, 1, 1, 300, 128, 0, [0, 41], [300, 257]),
    (5, 2, 2, 2, 64, 0, [0, 1, 4000, 64, 2000], [2, 1, 2, 0, 2]),    # split over many CTAs
    (1, 4, 1, 4, 128, 16, [3999], [4]),
    (4, 8, 8, 3, 128, 16, [4000, 3500, 129, 3900], [3, 2, 3, 1]),    # several tiles of several units a CTA
    (6, 6, 6, 2, 64, 8, [4000, 3500, 1290, 3900, 2200, 3000], [2, 2, 1, 2, 0, 2]),
    (4, 24, 6, 33, 128, 32, [2500, 1800, 2100, 40], [33, 32, 9, 33]),   # 132 rows: pairs
    (5, 20, 4, 26, 64, 0, [2500, 1800, 2100, 40, 1], [26, 25, 9, 26, 1]),
    # enough work for the small ranges that the CTAs take as they get done
    (4, 16, 8, 2, 128, 64, [8000, 7900, 8100, 7000], [2, 1, 2, 2]),
    (5, 8, 8, 3, 64, 0, [8000, 7900, 30, 8100, 7000], [3, 2, 3, 0, 1]),
    (80, 8, 8, 1, 64, 16, [400 + 3 * i for i in range(80)], [1] * 79 + [0]),   # more units than ranges
    (40, 4, 4, 2, 64, 32, [i * 17 % 300 for i in range(40)], [i % 3 for i in range(40)]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:6])))
def test_tree_parity(torch, eb, case):
    x = make(torch, *case, seed=sum(case[:6]))
    o, lse = call(torch, eb, x)
    assert eb.device_status() == 0
    check(torch, o, lse, want(x))
    o2, lse2 = call(torch, eb, x)          # the same bits again
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kind", ["chain", "roots"])
@pytest.mark.parametrize("d", [64, 128])
def test_tree_shapes(torch, eb, kind, d):
    x = make(torch, 2, 8, 2, 70, d, 16, [150, 37], [70, 66], seed=5, kind=kind)
    o, lse = call(torch, eb, x)
    check(torch, o, lse, want(x))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("std", [0.0, 30.0])
def test_tree_flat_and_steep_scores(torch, eb, d, std):
    """Equal scores, and scores of several hundred whose maximum moves from
    tile to tile."""
    x = make(torch, 2, 4, 2, 9, d, 16, [900, 402], [9, 5], seed=6, qstd=std)
    o, lse = call(torch, eb, x)
    check(torch, o, lse, want(x))


def test_tree_rising_scores(torch, eb):
    """Keys that grow along the cache: every tile passes the running maximum
    by far, so each one rescales."""
    x = make(torch, 1, 2, 1, 3, 128, 16, [1500], [3], seed=7)
    ramp = torch.linspace(0, 4, 1500)[None, :, None]
    x["k"][0] = (x["q"][0, 0, 0].float() * ramp).bfloat16()
    x["kc"] = torch.full_like(x["kc"], float("nan"))
    for j in range(-(-1500 // 16)):
        m = min(16, 1500 - 16 * j)
        x["kc"][int(x["table"][0, j]), :, :m] = x["k"][0][:, 16 * j:16 * j + m]
    o, lse = call(torch, eb, x)
    check(torch, o, lse, want(x))


@pytest.mark.parametrize("d", [64, 128])
def test_tree_nan_stays_in_its_row(torch, eb, d):
    """A query of NaN among live rows, over enough tiles that every CTA takes
    several: its row is NaN, the others are what they are without it."""
    x = make(torch, 4, 16, 8, 7, d, 16, [4000, 3500, 129, 3900], [7, 5, 7, 1], seed=16)
    w = want(x)
    x["q"][0, 3, 2] = float("nan")
    x["q"][3, 15, 0, 1] = float("nan")
    o, lse = call(torch, eb, x)
    o, lse = o.cpu(), lse.cpu()
    for b, h, i in [(0, 3, 2), (3, 15, 0)]:
        assert bool(torch.isnan(o[b, h, i]).all()) and bool(torch.isnan(lse[b, h, i]))
        o[b, h, i], lse[b, h, i] = w[0][b, h, i].to(o.dtype), w[1][b, h, i].float()
    check(torch, o, lse, w)


def test_tree_equals_paged_decode_for_a_chain(torch, eb):
    """A chain of drafts is multi-token decode with the same keys stored."""
    B, Hq, Hkv, N, d, ps = 3, 16, 4, 4, 128, 16
    L = [200, 31, 512]
    x = make(torch, B, Hq, Hkv, N, d, ps, L, [N] * B, seed=8, kind="chain")
    o, lse = call(torch, eb, x)
    # the same tokens through the page plan and the append
    mp = x["table"].shape[1] + 1
    table = np.full((B, mp), -1, np.int32)
    table[:, :mp - 1] = x["table"]
    pages = x["kc"].shape[0]
    kc = torch.cat([x["kc"], torch.zeros_like(x["kc"][:8])]).cuda()
    vc = torch.cat([x["vc"], torch.zeros_like(x["vc"][:8])]).cuda()
    kc, vc = kc.nan_to_num(0.0), vc.nan_to_num(0.0)
    ring = np.zeros(pages + 8, np.int32)
    ring[:8] = np.arange(pages, pages + 8)
    old, new = i32(torch, L), i32(torch, np.array(L) + N)
    td = i32(torch, table)
    slots, _ = eb.paged_plan(old, new, td, i32(torch, ring), i32(torch, [0, 8]), ps, N)
    eb.kv_append(x["kn"].cuda(), x["vn"].cuda(), slots, kc, vc)
    o2, lse2 = eb.attn_fwd_paged(x["q"].cuda(), kc, vc, td, new, causal=True)
    assert eb.device_status() == 0
    w = want(x)
    check(torch, o, lse, w)
    check(torch, o2, lse2, w)


def test_tree_bad_entries_are_reported(torch, eb):
    """Table entries outside the cache read as zeros, parents outside [-1, i)
    as -1; both are reported."""
    x = make(torch, 2, 4, 2, 6, 128, 16, [100, 90], [6, 6], seed=9)
    x["table"][1, 2] = 10 ** 6
    x["k"][1][:, 32:48] = 0
    x["v"][1][:, 32:48] = 0
    o, lse = call(torch, eb, x)
    assert eb.device_status() == 7
    check(torch, o, lse, want(x))
    x = make(torch, 1, 4, 2, 6, 64, 0, [40], [6], seed=10)
    x["parents"][0] = [-1, 1, 5, -7, 2, 2 ** 31 - 1]
    o, lse = call(torch, eb, x)
    assert eb.device_status() == 7
    check(torch, o, lse, want(x))


def test_tree_lengths_are_clamped(torch, eb):
    x = make(torch, 3, 4, 2, 6, 128, 0, [40, 40, 0], [6, 0, 6], seed=11, cap=40)
    w = want(x)
    x["L"] = np.array([1000, 40, -5], np.int32)
    x["n"] = np.array([2 ** 31 - 1, -3, 6], np.int32)
    o, lse = call(torch, eb, x)
    check(torch, o, lse, w)


def test_tree_without_optional_arguments(torch, eb):
    """key_lens and new_lens left out, lse not returned, a scale of one's
    own, buffers of the caller, another stream."""
    x = make(torch, 2, 4, 2, 6, 128, 0, [77, 77], [6, 6], seed=12)
    d = {k: x[k].cuda() for k in ("q", "kc", "vc", "kn", "vn")}
    par = i32(torch, x["parents"])
    out = torch.full_like(d["q"], 7.0)
    ws = torch.empty(eb.attn_tree_workspace_size(2, 4, 2, 6, 128), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = eb.attn_fwd_tree(d["q"], d["kc"], d["vc"], None, d["kn"], d["vn"], par, scale=0.25,
                           out=out, workspace=ws, return_lse=False, stream=s)
    s.synchronize()
    assert got is out
    w = want(x, 0.25)
    assert bool(((out.cpu().double() - w[0]).abs() <= w[2]).all())
    with pytest.raises(eb.AttnError) as e:
        eb.attn_fwd_tree(d["q"], d["kc"], d["vc"], None, d["kn"], d["vn"], par,
                         workspace=ws[:ws.numel() - 1])
    assert e.value.status == 4


def test_tree_graphs_share_a_workspace(torch, eb):
    """Two captured calls of different sizes on one workspace, replayed in
    turn with new inputs."""
    a = make(torch, 2, 8, 2, 16, 128, 16, [900, 333], [16, 9], seed=13)
    b = make(torch, 3, 4, 4, 5, 64, 0, [50, 800, 0], [5, 5, 2], seed=14)
    need = max(eb.attn_tree_workspace_size(2, 8, 2, 16, 128), eb.attn_tree_workspace_size(3, 4, 4, 5, 64))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graphs = []
    for x in (a, b):
        d = [x["q"].cuda(), x["kc"].cuda(), x["vc"].cuda(), i32(torch, x["L"]), x["kn"].cuda(),
             x["vn"].cuda(), i32(torch, x["parents"])]
        kw = dict(new_lens=i32(torch, x["n"]), workspace=ws,
                  block_table=None if x["table"] is None else i32(torch, x["table"]))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            eb.attn_fwd_tree(*d, **kw)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, lse = eb.attn_fwd_tree(*d, **kw)
        graphs.append((g, d, o, lse, x))
    for r in range(3):
        for g, d, o, lse, x in graphs:
            g.replay()
        for g, d, o, lse, x in graphs:
            check(torch, o, lse, want(x))
            x["q"] = torch.roll(x["q"], 1, 1)       # the heads' queries change places
            d[0].copy_(x["q"])


@pytest.mark.parametrize("case", [
    # B, Hq, Hkv, Nq, d, page size, cached lengths, nodes
    (2, 64, 1, 40, 64, 16, [300, 1000], [40, 33]),                       # 2560 rows: ten row groups
    (1, 1, 1, 1024, 64, 0, [100], [1024]),                               # the largest tree
    (2048, 1, 1, 2, 64, 8, [(i * 7) % 40 for i in range(2048)], [i % 3 for i in range(2048)]),
], ids=["rows", "nodes", "sequences"])
def test_tree_largest_counts(torch, eb, case):
    x = make(torch, *case, seed=17, kind="chain" if case[3] == 1024 else "random")
    o, lse = call(torch, eb, x)
    assert eb.device_status() == 0
    check(torch, o, lse, want(x))


@pytest.mark.parametrize("Hq", [4, 64])
def test_tree_output_on_a_16_byte_boundary(torch, eb, Hq):
    x = make(torch, 2, Hq, 4, 9, 128, 16, [90, 33], [9, 4], seed=18)
    n = x["q"].numel()
    out = torch.empty(n + 8, dtype=torch.bfloat16, device="cuda")[8:].view(x["q"].shape)
    assert out.data_ptr() % 32 == 16
    o, lse = call(torch, eb, x, out=out)
    check(torch, o, lse, want(x))


def test_tree_pages_past_4_gib(torch, eb):
    """Pages at the end of a 5 GiB pool."""
    Hkv, ps, d, pages = 8, 128, 128, 20480
    x = make(torch, 2, 8, Hkv, 3, d, ps, [300, 129], [3, 2], seed=19)
    kc = torch.empty(pages, Hkv, ps, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    table = x["table"].copy()
    for i, (b, j) in enumerate((b, j) for b in range(2) for j in range(table.shape[1]) if table[b, j] >= 0):
        p = pages - 1 - i
        kc[p], vc[p] = x["kc"][int(table[b, j])].cuda(), x["vc"][int(table[b, j])].cuda()
        x["table"][b, j] = p
    w = want(x)
    x["kc"], x["vc"] = kc, vc
    o, lse = call(torch, eb, x)
    assert eb.device_status() == 0
    check(torch, o, lse, w)


def test_tree_calls_on_two_streams(torch, eb):
    """Calls that overlap, each with a workspace of its own."""
    xs = [make(torch, 3, 8, 4, 16, 128, 16, [2000, 900, 1500], [16, 9, 12], seed=20),
          make(torch, 2, 16, 16, 25, 64, 0, [1800, 700], [25, 20], seed=21)]
    ws = [want(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    args = []
    for x in xs:
        d = [x["q"].cuda(), x["kc"].cuda(), x["vc"].cuda(), i32(torch, x["L"]), x["kn"].cuda(),
             x["vn"].cuda(), i32(torch, x["parents"])]
        args.append((d, dict(new_lens=i32(torch, x["n"]),
                             block_table=None if x["table"] is None else i32(torch, x["table"]))))
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for s, (d, kw) in zip(streams, args):
            outs.append(eb.attn_fwd_tree(*d, stream=s, **kw))
    torch.cuda.synchronize()
    assert eb.device_status() == 0
    for i, (o, lse) in enumerate(outs):
        check(torch, o, lse, ws[i % 2])


def test_steps_without_synchronising(torch, eb):
    """Forty steps of plan, append, tree attention and paged decode queued one
    behind the other give the bits of the same steps with a synchronisation
    after every call.  (The kernels start before their predecessors end; each
    one waits for all work before it.)  One sequence stays empty."""
    B, Hq, Hkv, N, d, ps, mp, pages = 3, 8, 2, 4, 128, 16, 20, 64

    def go(sync):
        g = torch.Generator(device="cuda")
        g.manual_seed(5)
        table = torch.full((B, mp), -1, dtype=torch.int32, device="cuda")
        ring = torch.arange(pages, dtype=torch.int32, device="cuda")
        state = torch.tensor([0, pages], dtype=torch.int32, device="cuda")
        kc = torch.zeros(pages, Hkv, ps, d, dtype=torch.bfloat16, device="cuda")
        vc = torch.zeros_like(kc)
        old = torch.zeros(B, dtype=torch.int32, device="cuda")
        par = torch.arange(-1, N - 1, dtype=torch.int32, device="cuda").repeat(B, 1)
        grow = torch.tensor([3, 0, 4], dtype=torch.int32, device="cuda")
        n = torch.tensor([4, 0, 4], dtype=torch.int32, device="cuda")
        outs = []
        wait = torch.cuda.synchronize if sync else (lambda: None)
        for _ in range(40):
            x = torch.randn(B, N, Hq + 2 * Hkv, d, generator=g, device="cuda").bfloat16().transpose(1, 2)
            pos = old[:, None] + torch.arange(N, dtype=torch.int32, device="cuda")
            wait()
            q, k = eb.kv_append(x[:, Hq:Hq + Hkv], q=x[:, :Hq], positions=pos)
            wait()
            v = x[:, Hq + Hkv:].contiguous()
            o, lse = eb.attn_fwd_tree(q, kc, vc, old, k, v, par, new_lens=n, block_table=table)
            wait()
            new = old + grow
            slots, state = eb.paged_plan(old, new, table, ring, state, ps, N)
            wait()
            eb.kv_append(k, v, slots, kc, vc)
            wait()
            empty = eb.attn_fwd_paged(q[:, :, :1].contiguous(), kc, vc, table, old * 0)[0]
            wait()
            o2, lse2 = eb.attn_fwd_paged(q[:, :, :1].contiguous(), kc, vc, table, new)
            outs += [o, lse, empty, o2, lse2]
            old = new
        torch.cuda.synchronize()
        assert eb.device_status() == 0
        return outs + [kc, vc, table, state]

    for a, b in zip(go(False), go(True)):
        assert torch.equal(a, b)


def test_verify_step(torch, eb):
    """Plan, append, tree attention and the paged decode together, as a server
    runs them: a prompt, then steps that draft a tree, verify it and store the
    accepted path; each step against the reference over the tokens so far."""
    rng = np.random.default_rng(15)
    B, Hq, Hkv, N, d, ps, mp, pages = 3, 8, 2, 11, 128, 16, 12, 40
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32)).bfloat16()
    table, ring, state = (i32(torch, np.full((B, mp), -1)), i32(torch, rng.permutation(pages)),
                          i32(torch, [7, pages]))
    nan = float("nan")
    kc = torch.full((pages, Hkv, ps, d), nan, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    old = np.zeros(B, np.int32)
    new = np.array([40, 1, 16], np.int32)
    Np = 40
    k, v = bf(B, Hkv, Np, d), bf(B, Hkv, Np, d)
    pos = np.tile(np.arange(Np), (B, 1)).astype(np.int32)
    slots, state = eb.paged_plan(i32(torch, old), i32(torch, new), table, ring, state, ps, Np)
    _, kr = eb.kv_append(k.cuda(), v.cuda(), slots, kc, vc, positions=i32(torch, pos), return_k=True)
    hist = [(kr[b, :, :new[b]].cpu(), v[b, :, :new[b]]) for b in range(B)]
    old = new
    for it in range(4):
        n = rng.integers(1, N + 1, B).astype(np.int32)
        par = random_tree(rng, B, N)
        depth = np.zeros((B, N), np.int32)
        for b in range(B):
            for i in range(N):
                depth[b, i] = 0 if par[b, i] < 0 else depth[b, par[b, i]] + 1
        x = bf(B, N, Hq + 2 * Hkv, d).transpose(1, 2)
        xc = x.cuda()
        q, kr = eb.kv_append(xc[:, Hq:Hq + Hkv], q=xc[:, :Hq],
                             positions=i32(torch, old[:, None] + depth))
        vn = xc[:, Hq + Hkv:].contiguous()
        o, lse = eb.attn_fwd_tree(q, kc, vc, i32(torch, old), kr, vn, i32(torch, par),
                                  new_lens=i32(torch, n), block_table=table)
        z = lambda t: t.cpu().double()
        w = ref.tree(z(q), [z(h[0]) for h in hist], [z(h[1]) for h in hist], old, z(kr), z(vn),
                     par, n, 1 / math.sqrt(d))
        check(torch, o, lse, w)
        # accept the path to a random node; sequence 1 finishes after the third step
        index = np.full((B, N), -1, np.int32)
        new = old.copy()
        for b in range(B):
            a = int(rng.integers(0, n[b]))
            new[b] = old[b] + depth[b, a] + 1
            path = []
            while a >= 0:
                index[b, a] = depth[b, a]
                path.append(a)
                a = par[b, a]
            path = path[::-1]
            hist[b] = (torch.cat([hist[b][0], kr[b][:, path].cpu()], 1),
                       torch.cat([hist[b][1], vn[b][:, path].cpu()], 1))
        if it == 2:
            new[1] = 0
            index[1] = -1
            hist[1] = (hist[1][0][:, :0], hist[1][1][:, :0])
        slots, state = eb.paged_plan(i32(torch, old), i32(torch, new), table, ring, state, ps, N,
                                     index=i32(torch, index))
        eb.kv_append(kr, vn, slots, kc, vc)
        old = new
    assert eb.device_status() == 0
    held = int((-(-old // ps)).sum())
    assert int(state[1]) == pages - held
    # the pages in use and in the queue are all there, once
    used = [int(table[b, j]) for b in range(B) for j in range(-(-old[b] // ps))]
    h, c = (int(s) for s in state)
    free = [int(ring[(h + m) % pages]) for m in range(c)]
    assert sorted(used + free) == list(range(pages))
