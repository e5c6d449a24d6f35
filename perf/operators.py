"""Cases of the paged-cache serving operators: the step's page plan (block
tables and slot maps from request lengths), storing and rotating new keys and
values, and attention for a tree of drafted tokens over a cache.

`own` selects what run() computes with: plain torch operations (False) or the
library's entry points (True)."""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
ROPE_BASE = 10000.0


# ------------------------------------------------------------------ cases

def listed():
    return [
        # -- page plan
        # one decode step of a full batch: one token each, a sixteenth of the sequences need a page
        dict(name="plan_decode", op="plan", B=256, N=1, ps=16, max_pages=1024, lo=1024, hi=16383,
             grow=1, free=0, index=False),
        # prompts admitted together, padded to the longest: every page and every slot is new
        dict(name="plan_prompts", op="plan", B=32, N=8192, ps=16, max_pages=1024, lo=0, hi=0,
             grow=8192, free=0, index=False),
        # after a verification: few of 63 drafted nodes accepted, one sequence in ten finished
        dict(name="plan_accept", op="plan", B=1000, N=63, ps=32, max_pages=128, lo=5, hi=4000,
             grow=6, free=10, index=True),
        # -- storing
        # decode step: one token per sequence, q and k rotated at its own position
        dict(name="append_decode", op="append", B=64, N=1, Hq=32, Hkv=8, d=128, ps=16, rope=True,
             pairing=0, fused=True, keep=100),
        # after a verification: the accepted few of 63 rotated nodes go to the cache
        dict(name="append_accept", op="append", B=64, N=63, Hq=0, Hkv=8, d=128, ps=16, rope=False,
             pairing=0, fused=False, keep=6),
        # prompts: 32768 tokens, views of a fused projection's output
        dict(name="append_prompt", op="append", B=4, N=8192, Hq=32, Hkv=8, d=128, ps=16, rope=True,
             pairing=0, fused=True, keep=100),
        # -- tree attention
        # one short chat, one token: latency
        dict(name="tree_single", op="tree", B=1, Hq=32, Hkv=8, d=128, N=1, nlo=1, lo=777, hi=777, ps=16),
        # draft verification of 16 sequences, 16 nodes each (64 rows per kv head)
        dict(name="tree_gqa", op="tree", B=16, Hq=32, Hkv=8, d=128, N=16, nlo=9, lo=1028, hi=16384, ps=16),
        # multi-query heads, short chains over a ragged cache (128 rows per kv head)
        dict(name="tree_mqa", op="tree", B=64, Hq=32, Hkv=1, d=128, N=4, nlo=4, lo=1024, hi=16384, ps=64),
        # d = 64 without head sharing, odd node counts, contiguous cache
        dict(name="tree_mha64", op="tree", B=8, Hq=16, Hkv=16, d=64, N=25, nlo=13, lo=2048, hi=4095, ps=0),
        # large trees over long caches (256 rows per kv head): both roofs near
        dict(name="tree_long", op="tree", B=8, Hq=32, Hkv=8, d=128, N=64, nlo=64, lo=8192, hi=32768, ps=128),
        # large trees on multi-query heads (2048 rows per kv head): tensor-bound
        dict(name="tree_wide", op="tree", B=16, Hq=32, Hkv=1, d=128, N=64, nlo=33, lo=4096, hi=16384, ps=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "tree", "tree"])
    if op == "plan":
        ps = rng.choice([8, 16, 32, 64, 128])
        N = _log(rng, 1, 8192)
        B = _log(rng, 1, min(2048, max(1, 262144 // N)))
        hi = rng.randint(0, 16384)
        grow = rng.choice([1, N, rng.randint(1, N)])
        max_pages = -(-(hi + grow + rng.randint(0, 500)) // ps)
        return dict(op="plan", B=B, N=N, ps=ps, max_pages=max_pages, lo=rng.randint(0, hi), hi=hi,
                    grow=grow, free=rng.choice([0, 0, 3, 10]), index=rng.random() < 0.4)
    if op == "append":
        d = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 4, 8])
        N = _log(rng, 1, 8192)
        B = _log(rng, 1, min(512, max(1, 32768 // N)))
        rope = rng.random() < 0.7
        fused = rng.random() < 0.5
        return dict(op="append", B=B, N=N, Hq=G * Hkv if rope else 0, Hkv=Hkv, d=d,
                    ps=rng.choice([8, 16, 32, 64]), rope=rope, pairing=rng.choice([0, 1]),
                    fused=fused, keep=rng.choice([100, 100, 50, 6]))
    while True:
        d = rng.choice([64, 128, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 4, 7, 8, 16])
        N = _log(rng, 1, 128)
        B = _log(rng, 1, 64)
        hi = _log(rng, 64, 32768)
        if B * Hkv * hi * d <= 2 ** 27 and B * Hkv * G * N * hi * d <= 2 ** 36:
            break
    ps = rng.choice([0, 8, 16, 32, 64, 128 if d == 128 else 64])
    return dict(op="tree", B=B, Hq=G * Hkv, Hkv=Hkv, d=d, N=N, nlo=rng.randint(1, N),
                lo=rng.randint(0, hi), hi=hi, ps=ps)


# ------------------------------------------------------------------ sizes fixed by the case

def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi], the larger end among them."""
    return [hi - ((hi - lo) * i) // n for i in range(n)]


def _plan_lens(c):
    old = _spread(c["lo"], c["hi"], c["B"])
    # growth: the tokens accepted this step (1 .. grow), or the prompts' lengths
    g = [1 + (c["grow"] - 1) * ((7 * i) % c["B"] + 1) // c["B"] for i in range(c["B"])]
    cap = c["max_pages"] * c["ps"]
    new = [min(o + x, cap) for o, x in zip(old, g)]
    if c["free"]:
        new = [0 if i % c["free"] == 0 else n for i, n in enumerate(new)]
    return old, new


def _tree_lens(c):
    L = _spread(c["lo"], c["hi"], c["B"])
    n = _spread(c["nlo"], c["N"], c["B"])
    n = [n[(5 * i) % c["B"]] if c["B"] % 5 else n[i] for i in range(c["B"])]
    return L, n


def _kept(c):
    """Tokens of every sequence that are stored (the first ones of a random order)."""
    return max(1, c["N"] * c["keep"] // 100)


def work(c):
    B, N = c["B"], c["N"]
    if c["op"] == "plan":
        old, new = _plan_lens(c)
        h = [(-(-o // c["ps"]), -(-n // c["ps"])) for o, n in zip(old, new)]
        pages = sum(abs(y - x) for x, y in h)
        return {"bytes": 8 * B + 16 + 8 * pages + 4 * B * N * (2 if c["index"] else 1), "flops": B * N}
    if c["op"] == "append":
        rows = B * N * c["Hkv"]
        kept = B * _kept(c) * c["Hkv"]
        row = 2 * c["d"]
        q = B * N * c["Hq"] * row
        by = 2 * q + 4 * B * N + kept * 4 * row
        if c["rope"]:
            by += 4 * B * N
            if c["keep"] < 100:                       # rotated keys also kept outside the cache
                by += (rows - kept) * row + rows * row
        return {"bytes": by, "flops": 3 * (B * N * c["Hq"] + rows) * c["d"] if c["rope"] else kept}
    L, n = _tree_lens(c)
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    by = sum(L) * Hkv * d * 4 + sum(n) * Hkv * d * 4            # cached and drafted keys and values
    by += sum(n) * Hq * d * 2 + B * N * Hq * (2 * d + 4)        # q, o, lse
    by += 4 * sum(n) + 8 * B
    if c["ps"]:
        by += sum(-(-x // c["ps"]) for x in L) * 4
    fl = sum(4 * Hq * y * (x + 1) * d for x, y in zip(L, n))
    return {"bytes": by, "flops": fl}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _bf16(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).bfloat16()


def _i32(x):
    return torch.tensor(np.asarray(x, np.int32), device=DEV)


def prepare(c, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    s = {"c": c}
    B, N = c["B"], c["N"]
    if c["op"] == "plan":
        old, new = _plan_lens(c)
        perm = rng.permutation(B)
        old, new = np.array(old)[perm], np.array(new)[perm]
        ps = c["ps"]
        held, want = -(-old // ps), -(-new // ps)
        need = int(np.maximum(want - held, 0).sum())
        num_pages = int(held.sum()) + need + 37          # some pages stay free
        ids = rng.permutation(num_pages).astype(np.int32)
        table = np.full((B, c["max_pages"]), -1, np.int32)
        at = 0
        for b in range(B):
            table[b, :held[b]] = ids[at:at + held[b]]
            at += held[b]
        free = ids[at:]
        head = int(rng.integers(0, num_pages))
        ring = np.full(num_pages, -1, np.int32)
        ring[(head + np.arange(len(free))) % num_pages] = free
        s.update(old=_i32(old), new=_i32(new), table=_i32(table), ring=_i32(ring),
                 state=_i32([head, len(free)]))
        s["index"] = None
        if c["index"]:
            # node -> place on the accepted path, -1 for a rejected node
            grow = np.maximum(new - old, 0)
            idx = np.full((B, N), -1, np.int32)
            for b in range(B):
                k = min(int(grow[b]), N)
                idx[b, np.sort(rng.choice(N, k, replace=False))] = np.arange(k)
            s["index"] = _i32(idx)
        return s
    if c["op"] == "append":
        Hq, Hkv, d, ps = c["Hq"], c["Hkv"], c["d"], c["ps"]
        if c["fused"]:      # q, k, v are views of the projection's output [B, N, heads * d]
            x = _bf16(g, B, N, (Hq + 2 * Hkv) * d).view(B, N, Hq + 2 * Hkv, d).transpose(1, 2)
            s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        else:
            s["q"], s["k"], s["v"] = (_bf16(g, B, h, N, d) for h in (Hq, Hkv, Hkv))
        if Hq == 0:
            s["q"] = None
        kept = _kept(c)
        num_pages = -(-B * kept // ps) + 2
        slot = rng.permutation(num_pages * ps)[:B * kept].astype(np.int32)
        if N >= 128:        # a prompt's tokens fill whole pages in order
            pages = rng.permutation(num_pages)
            flat = np.arange(B * kept)
            slot = (pages[flat // ps] * ps + flat % ps).astype(np.int32)
        slots = np.full((B, N), -1, np.int32)
        for b in range(B):
            slots[b, np.sort(rng.choice(N, kept, replace=False))] = slot[b * kept:(b + 1) * kept]
        s["slots"] = _i32(slots)
        s["kc"] = _bf16(g, num_pages, Hkv, ps, d)
        s["vc"] = _bf16(g, num_pages, Hkv, ps, d)
        s["pos"] = None
        if c["rope"]:
            start = rng.integers(0, 100000, B) if N < 128 else np.zeros(B, np.int64)
            s["pos"] = _i32(start[:, None] + np.arange(N)[None])
        return s
    Hq, Hkv, d, ps = c["Hq"], c["Hkv"], c["d"], c["ps"]
    L, n = _tree_lens(c)
    perm = rng.permutation(B)
    L, n = np.array(L)[perm], np.array(n)[perm]
    s["q"] = _bf16(g, B, Hq, N, d, std=2.0)
    s["kn"], s["vn"] = _bf16(g, B, Hkv, N, d), _bf16(g, B, Hkv, N, d)
    u = rng.random((B, N))
    s["parents"] = _i32(np.floor(u * (np.arange(N) + 1)) - 1)      # every node hangs on an earlier one
    s["L"], s["n"] = _i32(L), _i32(n)
    s["hostL"], s["hostn"] = [int(x) for x in L], [int(x) for x in n]
    if ps:
        held = -(-L // ps)
        mp = max(1, int(held.max()))
        num_pages = int(held.sum()) + 1
        ids = rng.permutation(num_pages).astype(np.int32)
        table = np.full((B, mp), -1, np.int32)
        at = 0
        for b in range(B):
            table[b, :held[b]] = ids[at:at + held[b]]
            at += held[b]
        s["table"] = _i32(table)
        s["kc"], s["vc"] = _bf16(g, num_pages, Hkv, ps, d), _bf16(g, num_pages, Hkv, ps, d)
    else:
        cap = max(1, int(L.max()))
        s["table"] = None
        s["kc"], s["vc"] = _bf16(g, B, Hkv, cap, d), _bf16(g, B, Hkv, cap, d)
    return s


# ------------------------------------------------------------------ plain forms

def _plan_plain(s):
    c = s["c"]
    ps, N, dev = c["ps"], c["N"], s["old"].device
    table, ring = s["table"], s["ring"]
    cap, P = table.shape[1] * ps, ring.numel()
    old, new = s["old"].long().clamp(0, cap), s["new"].long().clamp(0, cap)
    held, want = (old + ps - 1) // ps, (new + ps - 1) // ps
    take, give = (want - held).clamp(min=0), (held - want).clamp(min=0)
    head, count = s["state"][0].long(), s["state"][1].long()
    j = torch.arange(table.shape[1], device=dev)[None]
    # pages taken from the front of the free queue, in request order
    first = (take.cumsum(0) - take)[:, None] + j - held[:, None]
    taking = (j >= held[:, None]) & (j < want[:, None])
    page = torch.where(first < count, ring[((head + first) % P)].long(), -1)
    # pages given back to its end
    back = (give.cumsum(0) - give)[:, None] + j - want[:, None]
    giving = (j >= want[:, None]) & (j < held[:, None])
    at = torch.where(giving & (back < P - count), (head + count + back) % P, P)
    ext = torch.cat([ring, ring.new_zeros(1)])
    ext.scatter_(0, at.reshape(-1), table.reshape(-1))
    ring.copy_(ext[:P])
    table.copy_(torch.where(taking, page.int(), table))
    served = torch.minimum(take.sum(), count)
    state = torch.stack([(head + served) % P,
                         count - served + torch.minimum(give.sum(), P - count)]).int()
    t = torch.arange(N, device=dev)[None].expand(c["B"], N) if s["index"] is None else s["index"].long()
    pos = old[:, None] + t
    ok = (t >= 0) & (t < (new - old)[:, None])
    pg = table.long().gather(1, torch.where(ok, pos // ps, 0))
    slots = torch.where(ok & (pg >= 0) & (pg < P), pg * ps + pos % ps, -1).int()
    return slots, state, table, ring


def _rotate_plain(x, pos, pairing):
    d = x.shape[-1]
    theta = ROPE_BASE ** (-2.0 * torch.arange(d // 2, device=x.device, dtype=torch.float64) / d)
    ang = pos.double()[:, None, :, None] * theta               # angles of far positions need 64 bits
    cos, sin = ang.cos().float(), ang.sin().float()
    x = x.float()
    if pairing == 0:
        a, b = x[..., :d // 2], x[..., d // 2:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)


def _store(cache, rows, slots, ps):
    """rows [B, Hkv, N, d] to the cache [pages, Hkv, ps, d] at slots [B, N] (-1: none)."""
    ok = slots >= 0
    sl = slots[ok].long()
    cache[sl // ps, :, sl % ps] = rows.transpose(1, 2)[ok].to(cache.dtype)


def _append_plain(s):
    c = s["c"]
    q, k = s["q"], s["k"]
    if c["rope"]:
        k = _rotate_plain(k, s["pos"], c["pairing"]).bfloat16()
        q = _rotate_plain(q, s["pos"], c["pairing"]).bfloat16()
    _store(s["kc"], k, s["slots"], c["ps"])
    _store(s["vc"], s["v"], s["slots"], c["ps"])
    return _append_outputs(s, q, k)


def _append_outputs(s, q, k):
    c = s["c"]
    out = [s["kc"], s["vc"]]
    if c["rope"]:
        out.append(q)
        if c["keep"] < 100:
            out.append(k)
    return out


def _ancestors(parents):
    """[B, N, N] truth values: node j is node i or one of its ancestors."""
    B, N = parents.shape
    m = torch.eye(N, device=parents.device).repeat(B, 1, 1)
    step = m + (parents[:, :, None] == torch.arange(N, device=parents.device)).float()
    for _ in range(max(1, math.ceil(math.log2(N + 1)))):
        step = ((step @ step) > 0).float()
    return step > 0


def _cached(cache, new, table):
    """The cache's and the drafts' rows of every sequence, [B, Hkv, capacity + N, d] in 32 bits."""
    if table is not None:
        x = cache[table.long().clamp(min=0)]                   # [B, pages, Hkv, ps, d]
        cache = x.transpose(1, 2).flatten(2, 3)
    return torch.cat([cache, new], 2).float()


def _tree_plain(s):
    c = s["c"]
    B, N, Hq, Hkv, d = c["B"], c["N"], c["Hq"], c["Hkv"], c["d"]
    k, v = _cached(s["kc"], s["kn"], s["table"]), _cached(s["vc"], s["vn"], s["table"])
    cap = k.shape[2] - N
    node = torch.arange(N, device=DEV)
    live = node < s["n"][:, None]                              # [B, N]
    see = torch.cat([(torch.arange(cap, device=DEV) < s["L"][:, None])[:, None].expand(B, N, cap),
                     _ancestors(s["parents"])], 2) & live[:, :, None]
    x = s["q"].float().view(B, Hkv, -1, d) @ k.transpose(2, 3) / math.sqrt(d)
    x = x.view(B, Hq, N, cap + N).masked_fill_(~see[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = m.masked_fill(m == -math.inf, 0.0)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, -1, cap + N) @ v).view(B, Hq, N, d) / l.masked_fill(l == 0, 1.0)
    return o.bfloat16(), (m + l.log())[..., 0]


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["c"]
    if not own:
        return {"plan": _plan_plain, "append": _append_plain, "tree": _tree_plain}[c["op"]](s)
    import exact_scaled_dot_fwd_b200 as eb
    if c["op"] == "plan":
        slots, state = eb.paged_plan(s["old"], s["new"], s["table"], s["ring"], s["state"], c["ps"],
                                     c["N"], index=s["index"])
        return slots, state, s["table"], s["ring"]
    if c["op"] == "append":
        q, k = eb.kv_append(s["k"], s["v"], s["slots"], s["kc"], s["vc"], q=s["q"], positions=s["pos"],
                            rope_base=ROPE_BASE, rope_pairing=c["pairing"],
                            return_k=c["rope"] and c["keep"] < 100)
        return _append_outputs(s, q, k)
    return eb.attn_fwd_tree(s["q"], s["kc"], s["vc"], s["L"], s["kn"], s["vn"], s["parents"],
                            new_lens=s["n"], block_table=s["table"])


# ------------------------------------------------------------------ from the definition, 64 bits

def _exact_tree(s):
    """Row by row of the tree: each node's own list of keys, one sequence at a time."""
    c = s["c"]
    B, N, Hq, Hkv, d, ps = c["B"], c["N"], c["Hq"], c["Hkv"], c["d"], c["ps"]
    o = torch.zeros(B, Hq, N, d, dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq, N), -math.inf, dtype=torch.float64, device=DEV)
    parents = s["parents"].cpu().numpy()
    kv_of = torch.arange(Hq, device=DEV) // (Hq // Hkv)
    for b in range(B):
        L, n = s["hostL"][b], s["hostn"][b]
        if s["table"] is None:
            kc, vc = s["kc"][b, :, :L].double(), s["vc"][b, :, :L].double()
        else:
            j = torch.arange(L, device=DEV)
            page, off = s["table"][b].long()[j // ps], j % ps
            kc = s["kc"][page, :, off].double().transpose(0, 1)
            vc = s["vc"][page, :, off].double().transpose(0, 1)
        paths = []
        for i in range(n):
            path, a = [], i
            while a >= 0:
                path.append(a)
                a = int(parents[b, a])
            paths.append(path)
        see = torch.zeros(n, N, dtype=torch.bool)
        for i, path in enumerate(paths):
            see[i, path] = True
        see = see.to(DEV)
        for g in range(Hkv):                       # the heads that share kv head g
            heads = (kv_of == g).nonzero()[:, 0]
            qh = s["q"][b, heads, :n].double() / math.sqrt(d)
            xc = qh @ kc[g].T
            xn = torch.where(see, qh @ s["kn"][b, g].double().T, -math.inf)
            top = xn.amax(2)
            if L:
                top = torch.maximum(top, xc.amax(2))
            pc, pn = torch.exp(xc - top[..., None]), torch.exp(xn - top[..., None])
            total = pc.sum(2) + pn.sum(2)
            o[b, heads, :n] = (pc @ vc[g] + pn @ s["vn"][b, g].double()) / total[..., None]
            lse[b, heads, :n] = top + torch.log(total)
    return o, lse


def _exact_append(s):
    c = s["c"]
    d, ps = c["d"], c["ps"]

    def turn(x):
        i = torch.arange(d // 2, device=DEV, dtype=torch.float64)
        ang = s["pos"].double()[..., None] * torch.exp(i * (-2.0 / d) * math.log(ROPE_BASE))
        z = torch.polar(torch.ones_like(ang), ang)[:, None]
        x = x.double()
        if c["pairing"] == 0:
            w = torch.complex(x[..., :d // 2].contiguous(), x[..., d // 2:].contiguous()) * z
            return torch.cat([w.real, w.imag], -1)
        w = torch.view_as_complex(x.reshape(*x.shape[:-1], d // 2, 2).contiguous()) * z
        return torch.view_as_real(w).flatten(-2)

    k = turn(s["k"]) if c["rope"] else s["k"].double()
    q = turn(s["q"]) if c["rope"] else None
    kc, vc = s["kc"].double(), s["vc"].double()
    for b in range(c["B"]):
        t = (s["slots"][b] >= 0).nonzero()[:, 0]
        sl = s["slots"][b][t].long()
        page, off = sl // ps, sl % ps
        for h in range(c["Hkv"]):
            kc[page, h, off] = k[b, h, t]
            vc[page, h, off] = s["v"][b, h, t].double()
    out = [kc, vc]
    if c["rope"]:
        out.append(q)
        if c["keep"] < 100:
            out.append(k)
    return out


def _exact_plan(s):
    """One request, one page, one token at a time."""
    c = s["c"]
    ps, N = c["ps"], c["N"]
    old, new, table, ring = (s[n].cpu().numpy().copy() for n in ("old", "new", "table", "ring"))
    head, count = (int(x) for x in s["state"].cpu())
    P, cap = len(ring), table.shape[1] * ps
    taken = given = 0
    slots = np.full((c["B"], N), -1, np.int32)
    index = None if s["index"] is None else s["index"].cpu().numpy()
    for b in range(c["B"]):
        o, n = min(max(int(old[b]), 0), cap), min(max(int(new[b]), 0), cap)
        have, want = -(-o // ps), -(-n // ps)
        for j in range(have, want):
            table[b, j] = ring[(head + taken) % P] if taken < count else -1
            taken += 1
        for j in range(want, have):
            if given < P - count:
                ring[(head + count + given) % P] = table[b, j]
            given += 1
        t = np.arange(N) if index is None else index[b]
        ok = (t >= 0) & (t < n - o)
        p = o + t[ok]
        page = table[b, p // ps]
        slots[b, ok] = np.where((page >= 0) & (page < P), page * ps + p % ps, -1)
    served = min(taken, count)
    state = np.array([(head + served) % P, count - served + min(given, P - count)], np.int32)
    return slots, state, table, ring


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "plan":
        return _exact_plan(s)
    if c["op"] == "append":
        return _exact_append(s)
    return _exact_tree(s)
