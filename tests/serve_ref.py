"""64-bit references of the serving operators (page plan, cache append, tree
attention), written from their definitions, and the error bounds the tests
hold the kernels to.  A bf16 rounding is off by at most 2^-8 of the value, an
fp32 one by 2^-24."""
import math

import numpy as np
import torch

U16, U32 = 2.0 ** -8, 2.0 ** -24


def plan(old, new, table, ring, state, ps, N, index=None):
    """One request, one page, one token at a time.  Returns (slots, state,
    table, ring, bad): bad = a shortage, an overflow or an entry a slot could
    not use."""
    table, ring = table.copy(), ring.copy()
    P, cap = len(ring), table.shape[1] * ps
    head, count = int(state[0]) % P, min(max(int(state[1]), 0), P)
    B = len(old)
    slots = np.full((B, N), -1, np.int32)
    taken = given = 0
    bad = False
    for b in range(B):
        o, n = (min(max(int(x), 0), cap) for x in (old[b], new[b]))
        have, want = -(-o // ps), -(-n // ps)
        for j in range(have, want):
            table[b, j] = ring[(head + taken) % P] if taken < count else -1
            taken += 1
        for j in range(want, have):
            if given < P - count:
                ring[(head + count + given) % P] = table[b, j]
            given += 1
        for i in range(N):
            t = i if index is None else int(index[b, i])
            if 0 <= t < n - o:
                p = o + t
                page = int(table[b, p // ps])
                if 0 <= page < P:
                    slots[b, i] = page * ps + p % ps
                else:
                    bad = True
    bad |= taken > count or given > P - count
    served = min(taken, count)
    state = np.array([(head + served) % P, count - served + min(given, P - count)], np.int32)
    return slots, state, table, ring, bad


def rotate(x, positions, base, pairing):
    """x float64 [B, H, N, d] rotated at positions [B, N]."""
    d = x.shape[-1]
    theta = np.float64(np.float32(base)) ** (-2.0 * np.arange(d // 2) / d)
    ang = torch.from_numpy(positions.astype(np.float64)[..., None] * theta)[:, None]
    c, s = ang.cos(), ang.sin()
    y = x.clone()
    i = slice(0, d // 2) if pairing == 0 else slice(0, d, 2)
    j = slice(d // 2, d) if pairing == 0 else slice(1, d, 2)
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., i] * s + x[..., j] * c
    return y


def rotate_bound(x, y, pairing):
    """|error| of a rotated bf16 row: the output's rounding, and cos, sin, two
    products and a sum in fp32 (five roundings, of |a| + |b| at most)."""
    d = x.shape[-1]
    m = x.abs()
    if pairing == 0:
        m = m[..., :d // 2] + m[..., d // 2:]
        m = torch.cat([m, m], -1)
    else:
        m = (m[..., 0::2] + m[..., 1::2]).repeat_interleave(2, -1)
    return U16 * y.abs() + 5 * (1 + U16) * U32 * m


def tree(q, k, v, L, kn, vn, parents, n, scale):
    """float64 tensors; k, v: per sequence [Hkv, >= L, d].  Returns o, lse and
    their error bounds, computed row by row.

    Bounds: a score is a sum of d products in fp32 (d roundings), scaled to
    log2 units (two more) and raised (exp2: 2 units of 2^-23): es in all, as a
    relative error of the weight.  A weight is rounded to bf16 for the
    product with V, the sums of weights and of products have at most one
    rounding per key, O one to bf16 at the end."""
    B, Hq, N, d = q.shape
    Hkv = kn.shape[1]
    G = Hq // Hkv
    o = torch.zeros(B, Hq, N, d, dtype=torch.float64)
    lse = torch.full((B, Hq, N), -math.inf, dtype=torch.float64)
    to, tl = torch.zeros_like(o), torch.zeros(B, Hq, N, dtype=torch.float64)
    for b in range(B):
        Lb, nb = int(L[b]), int(n[b])
        for i in range(min(nb, N)):
            path, a = [], i
            while a >= 0:
                path.append(a)
                p = int(parents[b, a])
                a = p if -1 <= p < a else -1
            for g in range(Hkv):
                K = torch.cat([k[b][g, :Lb], kn[b, g, path]])
                V = torch.cat([v[b][g, :Lb], vn[b, g, path]])
                Q = q[b, g * G:(g + 1) * G, i]
                s = Q @ K.T * scale
                m = s.amax(1, keepdim=True)
                p = (s - m).exp()
                l = p.sum(1, keepdim=True)
                rows = slice(g * G, (g + 1) * G)
                o[b, rows, i] = p @ V / l
                lse[b, rows, i] = (m + l.log())[:, 0]
                top = s.abs().amax(1, keepdim=True)
                es = ((d * U32) * (Q.abs() @ K.abs().T * scale).amax(1, keepdim=True)
                      + 4 * U32 * 2 * top + 8 * U32)
                sums = len(K) * U32
                mean = p @ V.abs() / l
                rel = U16 + 2 * es + 2 * sums
                to[b, rows, i] = rel * (1 + U16) * mean + U16 * o[b, rows, i].abs() + 1e-30
                tl[b, rows, i] = (es + sums + 4 * U32 * (1 + lse[b, rows, i][:, None].abs()))[:, 0]
    return o, lse, to, tl
