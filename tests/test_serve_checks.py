"""The serving operators' refusals (paged_plan, kv_append, attn_fwd_tree):
argument checks of the C ABI and of the binding, on the CPU, before any CUDA
call."""
import ctypes

import pytest
import torch

import exact_scaled_dot_fwd_b200 as eb

P = ctypes.c_void_p(0x10000)      # aligned, never dereferenced
U = ctypes.c_void_p(0x10002)      # misaligned
OK, EINVAL, EUNSUP, EALIGN, EWS, ECUDA = 0, 1, 2, 3, 4, 5


def at(k):
    """Distinct aligned addresses, 1 GB apart."""
    return ctypes.c_void_p((k + 1) << 30)


@pytest.fixture(scope="module")
def L():
    from exact_scaled_dot_fwd_b200 import build
    build.build()
    return eb.lib()


def plan(L, **kw):
    a = dict(old=at(0), new=at(1), table=at(2), ring=at(3), state=at(4), out=at(5), index=None,
             slots=at(6), B=2, N=4, max_pages=8, ps=16, pages=32)
    a.update(kw)
    return L.paged_plan(a["old"], a["new"], a["table"], a["ring"], a["state"], a["out"], a["index"],
                        a["slots"], a["B"], a["N"], a["max_pages"], a["ps"], a["pages"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(old=None), EINVAL), (dict(new=None), EINVAL), (dict(table=None), EINVAL),
    (dict(ring=None), EINVAL), (dict(state=None), EINVAL), (dict(out=None), EINVAL),
    (dict(slots=None), EINVAL), (dict(B=0), EINVAL), (dict(N=0), EINVAL), (dict(ps=0), EINVAL),
    (dict(max_pages=0), EINVAL), (dict(pages=-1), EINVAL),
    (dict(out=at(4)), EINVAL),                                  # the state in place
    (dict(out=ctypes.c_void_p((5 << 30) + 4)), EINVAL),         # half in place
    (dict(max_pages=1 << 20, ps=1 << 11), EUNSUP), (dict(pages=1 << 27), EUNSUP),
    (dict(B=1 << 16, N=1 << 15), EUNSUP), (dict(slots=U), EALIGN), (dict(index=U), EALIGN),
])
def test_paged_plan_refusals(L, kw, rc):
    assert plan(L, **kw) == rc


def append(L, strides=None, **kw):
    a = dict(q=at(0), k=at(1), v=at(2), pos=at(3), base=1e4, pairing=0, qo=at(4), ko=at(5),
             slots=at(6), kc=at(7), vc=at(8), B=2, Hq=4, Hkv=2, N=8, d=128, ps=16, pages=32)
    a.update(kw)
    s = None if strides is None else (ctypes.c_int64 * 9)(*strides)
    return L.kv_append(a["q"], a["k"], a["v"], s, a["pos"], a["base"], a["pairing"], a["qo"],
                       a["ko"], a["slots"], a["kc"], a["vc"], a["B"], a["Hq"], a["Hkv"], a["N"],
                       a["d"], a["ps"], a["pages"], None)


FUSED = [8 * 1024, 128, 1024] * 3     # views of a projection's output, 1024 wide


@pytest.mark.parametrize("kw,rc", [
    (dict(k=None), EINVAL), (dict(q=None), EINVAL), (dict(q=None, Hq=0), EINVAL),
    (dict(qo=None), EINVAL), (dict(v=None), EINVAL), (dict(slots=None), EINVAL),
    (dict(kc=None), EINVAL), (dict(vc=None), EINVAL), (dict(ps=0), EINVAL), (dict(pages=0), EINVAL),
    (dict(pos=None), EINVAL),                                        # q without positions
    (dict(pos=None, q=None, Hq=0, qo=None), EINVAL),                 # rotated k without
    (dict(slots=None, v=None, kc=None, vc=None, ko=None), EINVAL),   # nothing to do
    (dict(base=0.0), EINVAL), (dict(base=float("nan")), EINVAL), (dict(pairing=2), EINVAL),
    (dict(N=0), EINVAL), (dict(B=-1), EINVAL), (dict(Hkv=0), EINVAL),
    (dict(d=96), EUNSUP), (dict(d=256), EUNSUP), (dict(pages=1 << 27), EUNSUP),
    (dict(pages=1 << 26, Hkv=2), EUNSUP), (dict(B=1 << 16, N=1 << 15), EUNSUP),
    (dict(Hq=1 << 16), EUNSUP),
    (dict(q=U), EALIGN), (dict(kc=U), EALIGN), (dict(slots=U), EALIGN), (dict(pos=U), EALIGN),
    (dict(strides=[8 * 1024, 128, 1028] + FUSED[3:]), EALIGN),
    (dict(strides=[8 * 1024, 128, -1024] + FUSED[3:]), EINVAL),
    (dict(qo=at(1)), EINVAL),                                        # q_out on k
    (dict(ko=at(4)), EINVAL),                                        # k_out on q_out
    (dict(kc=at(8)), EINVAL),                                        # one cache for both
    (dict(qo=at(0), strides=FUSED), EINVAL),                         # in place on a view
    (dict(qo=ctypes.c_void_p((1 << 30) + 256)), EINVAL),             # partial overlap
])
def test_kv_append_refusals(L, kw, rc):
    kw = dict(kw)
    assert append(L, kw.pop("strides", None), **kw) == rc


def tree(L, **kw):
    a = dict(q=P, kc=P, vc=P, table=P, mp=4, ps=16, pages=64, kn=P, vn=P, parents=P, n=None, o=P,
             lse=None, B=2, Hq=4, Hkv=2, Nq=8, Nk=0, d=128, scale=0.1, kl=P, ws=None, wsb=0)
    a.update(kw)
    return L.attn_fwd_tree(a["q"], a["kc"], a["vc"], a["table"], a["mp"], a["ps"], a["pages"],
                           a["kn"], a["vn"], a["parents"], a["n"], a["o"], a["lse"], a["B"],
                           a["Hq"], a["Hkv"], a["Nq"], a["Nk"], a["d"], a["scale"], a["kl"],
                           a["ws"], a["wsb"], None)


CONTIG = dict(table=None, mp=0, ps=0, pages=0, Nk=100)


@pytest.mark.parametrize("kw,rc", [
    (dict(q=None), EINVAL), (dict(kn=None), EINVAL), (dict(vn=None), EINVAL),
    (dict(parents=None), EINVAL), (dict(kl=None), EINVAL), (dict(o=None), EINVAL),
    (dict(Nk=64), EINVAL), (dict(mp=0), EINVAL), (dict(pages=0), EINVAL),
    (dict(table=None, Nk=100), EINVAL), (dict(CONTIG, Nk=0), EINVAL),
    (dict(Hq=3), EINVAL), (dict(scale=0.0), EINVAL), (dict(scale=float("inf")), EINVAL),
    (dict(Nq=0), EINVAL), (dict(d=96), EUNSUP), (dict(Nq=1025), EUNSUP), (dict(B=2049), EUNSUP),
    (dict(ps=12), EUNSUP), (dict(ps=256), EUNSUP), (dict(ps=48), EUNSUP),
    (dict(mp=1 << 27), EUNSUP), (dict(pages=1 << 26), EUNSUP),
    (dict(CONTIG, B=1024, Hkv=4, Nk=1 << 19), EUNSUP),
    (dict(kn=U), EALIGN), (dict(lse=U), EALIGN), (dict(parents=U), EALIGN),
])
def test_attn_fwd_tree_refusals(L, kw, rc):
    assert tree(L, **kw) == rc


def test_attn_fwd_tree_needs_a_workspace(L):
    # (the workspace's size needs a device: without one the call fails there)
    assert tree(L) in (EWS, ECUDA)
    assert tree(L, **CONTIG) in (EWS, ECUDA)
    assert L.attn_tree_workspace_size(2, 3, 2, 8, 128) == 0
    assert L.attn_tree_workspace_size(2, 4, 2, 8, 96) == 0
    assert L.attn_tree_workspace_size(2, 4, 2, 1025, 128) == 0


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_paged_plan_binding():
    good = [i32(3), i32(3), i32(3, 4), i32(10), i32(2)]
    with pytest.raises(ValueError, match="CUDA device"):
        eb.paged_plan(*good, 16, 5)
    for k, bad, err in [(0, i32(2), ValueError), (1, i32(4), ValueError),
                        (2, i32(3, 4).long(), TypeError), (3, i32(2, 5), ValueError),
                        (4, i32(3), ValueError), (2, i32(4, 3).T, ValueError)]:
        x = list(good)
        x[k] = bad
        with pytest.raises(err):
            eb.paged_plan(*x, 16, 5)
    with pytest.raises(ValueError, match="index has shape"):
        eb.paged_plan(*good, 16, 5, index=i32(3, 4))
    with pytest.raises(ValueError, match="slots has shape"):
        eb.paged_plan(*good, 16, 5, slots=i32(3, 6))
    with pytest.raises(ValueError, match="state_out has shape"):
        eb.paged_plan(*good, 16, 5, state_out=i32(1))


def test_kv_append_binding():
    k, v, q, c = bf16(2, 2, 5, 64), bf16(2, 2, 5, 64), bf16(2, 4, 5, 64), bf16(7, 2, 16, 64)
    s, p = i32(2, 5), i32(2, 5)
    with pytest.raises(ValueError, match="CUDA device"):
        eb.kv_append(k, v, s, c, c.clone(), q=q, positions=p)
    for args, kw, match in [
            ((k, None, s, c, c), {}, "go together"),
            ((k, v, s, c, None), {}, "go together"),
            ((k, v, s, c, c), dict(q=q), "needs positions"),
            ((k, v, s, c, c), dict(return_k=True), "needs positions"),
            ((k,), {}, "needs positions"),
            ((k, v, s, c, c), dict(q_out=q), "q_out without q"),
            ((k, v[:, :1], s, c, c), {}, "v has shape"),
            ((k, v, s[:, :4].contiguous(), c, c), {}, "slots has shape"),
            ((k, v, s, bf16(7, 3, 16, 64), bf16(7, 3, 16, 64)), {}, "does not match"),
            ((k, v, s, c, bf16(7, 2, 8, 64)), {}, "v_cache has shape"),
            ((k, v, s, c, c), dict(q=bf16(2, 4, 6, 64), positions=p), "shape mismatch"),
            ((k, v, s, c, c), dict(positions=i32(2, 4)), "positions has shape"),
            ((k.transpose(2, 3).contiguous().transpose(2, 3), v, s, c, c), {}, "last dimension"),
            ((k, v, s, c, c), dict(positions=p, k_out=bf16(2, 2, 5, 32)), "k_out has shape")]:
        with pytest.raises(ValueError, match=match):
            eb.kv_append(*args, **kw)
    with pytest.raises(TypeError):
        eb.kv_append(k.half(), v, s, c, c)
    with pytest.raises(TypeError):
        eb.kv_append(k, v, s.long(), c, c)


def test_attn_fwd_tree_binding():
    q, kn, c = bf16(2, 4, 5, 64), bf16(2, 2, 5, 64), bf16(2, 2, 30, 64)
    par, kl, tb = i32(2, 5), i32(2), i32(2, 3)
    pc = bf16(9, 2, 16, 64)
    with pytest.raises(ValueError, match="CUDA device"):
        eb.attn_fwd_tree(q, c, c, kl, kn, kn, par)
    with pytest.raises(ValueError, match="CUDA device"):
        eb.attn_fwd_tree(q, pc, pc, kl, kn, kn, par, block_table=tb, new_lens=kl)
    for args, kw, match in [
            ((q, c, c, kl, kn, bf16(2, 2, 4, 64), par), {}, "shape mismatch"),
            ((q, c, bf16(2, 2, 31, 64), kl, kn, kn, par), {}, "cache shapes"),
            ((q, bf16(2, 1, 30, 64), bf16(2, 1, 30, 64), kl, kn, kn, par), {}, "cache shapes"),
            ((q, pc, pc, kl, kn, kn, par), {}, "9 sequences"),
            ((q, pc, pc, None, kn, kn, par), dict(block_table=tb), "needs key_lens"),
            ((q, pc, pc, kl, kn, kn, par), dict(block_table=i32(3, 3)), "3 rows"),
            ((q, c, c, i32(3), kn, kn, par), {}, "3 entries"),
            ((q, c, c, kl, kn, kn, i32(2, 4)), {}, "parents has shape"),
            ((q, c, c, kl, kn, kn, par), dict(new_lens=i32(1)), "new_lens has shape"),
            ((q, c, c, kl, kn, kn, par), dict(out=bf16(2, 4, 4, 64)), "out has shape"),
            ((q[:, :, ::2], c, c, kl, kn, kn, par), {}, "contiguous")]:
        with pytest.raises(ValueError, match=match):
            eb.attn_fwd_tree(*args, **kw)
    with pytest.raises(TypeError):
        eb.attn_fwd_tree(q, c, c, kl, kn, kn, par.long())


def test_arguments_that_are_not_tensors():
    good = [i32(3), i32(3), i32(3, 4), i32(10), i32(2)]
    for k in range(5):
        x = list(good)
        x[k] = [1, 2, 3]
        with pytest.raises(TypeError, match="must be a torch.Tensor"):
            eb.paged_plan(*x, 16, 5)
    k, c, s = bf16(2, 2, 5, 64), bf16(7, 2, 16, 64), i32(2, 5)
    for args in [(1, k, s, c, c), (k, 1, s, c, c), (k, k, [1], c, c), (k, k, s, 1, c), (k, k, s, c, 1)]:
        with pytest.raises(TypeError, match="must be a torch.Tensor"):
            eb.kv_append(*args)
    q, kn, c, par, kl = bf16(2, 4, 5, 64), bf16(2, 2, 5, 64), bf16(2, 2, 30, 64), i32(2, 5), i32(2)
    good = [q, c, c, kl, kn, kn, par]
    for k in range(7):
        x = list(good)
        x[k] = [1, 2]
        with pytest.raises(TypeError, match="must be a torch.Tensor"):
            eb.attn_fwd_tree(*x)
    for kw in (dict(block_table=3), dict(new_lens=3), dict(out=3), dict(lse=3), dict(workspace=3)):
        with pytest.raises(TypeError, match="must be a torch.Tensor"):
            eb.attn_fwd_tree(*good, **kw)
