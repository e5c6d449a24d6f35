"""exact_scaled_dot_fwd_b200 -- exact scaled dot-product attention forward on
B200 (sm_100a).

Thin Python binding over the C ABI of libattn_b200.so (include/attn.h).  It
only marshals arguments: torch tensors supply device pointers and the current
CUDA stream; every step of the computation runs in the library's kernels.
There is no CPU or library fallback: if the shared library is missing or a
call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import math
import os

__all__ = ["attn_fwd", "attn_fwd_ws", "attn_workspace_size", "attn_set_workspace",
           "attn_fwd_paged", "attn_fwd_rope", "attn_fwd_decode_static", "rope_apply",
           "paged_plan", "kv_append", "attn_fwd_tree", "attn_tree_workspace_size",
           "prefill_tile_shape", "tile_plan", "prefill_trace", "device_status", "attn_last_device_status",
           "AttnError", "lib", "STATUS_NAMES"]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libattn_b200.so")

STATUS_NAMES = {0: "ATTN_OK", 1: "ATTN_EINVAL", 2: "ATTN_EUNSUPPORTED", 3: "ATTN_EALIGN",
                4: "ATTN_EWORKSPACE", 5: "ATTN_ECUDA", 6: "ATTN_ETIMEOUT", 7: "ATTN_ERANGE"}

_lib = None


class AttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)}")


def lib():
    """Load libattn_b200.so (raises OSError when it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise OSError(f"{LIB_PATH} is missing: build it with "
                          "`python -m exact_scaled_dot_fwd_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.attn_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, vp, vp]
        L.attn_fwd.restype = i
        L.attn_fwd_ws.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, vp, vp, sz, vp]
        L.attn_fwd_ws.restype = i
        L.attn_fwd_window.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, f, vp, vp, sz,
                                      vp]
        L.attn_fwd_window.restype = i
        L.attn_fwd_ex.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, f, vp, vp, sz, vp]
        L.attn_fwd_ex.restype = i
        L.attn_fwd_paged.argtypes = [vp, vp, vp, vp, i, i, i, vp, vp, i, i, i, i, i, i, i, f, vp,
                                     vp, sz, vp]
        L.attn_fwd_paged.restype = i
        L.attn_fwd_rope.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, vp, f, i, i, vp, sz,
                                    vp]
        L.attn_fwd_rope.restype = i
        L.attn_rope_workspace_size.argtypes = [i, i, i, i, i, i]
        L.attn_rope_workspace_size.restype = sz
        L.attn_workspace_size.argtypes = [i, i, i, i, i, i]
        L.attn_workspace_size.restype = sz
        L.attn_set_workspace.argtypes = [vp, sz]
        L.attn_set_workspace.restype = i
        L.rope_apply.argtypes = [vp, vp, i, i, i, i, f, i, i, vp]
        L.rope_apply.restype = i
        L.attn_prefill_tile_shape.argtypes = [i, ctypes.POINTER(i), ctypes.POINTER(i)]
        L.attn_prefill_tile_shape.restype = i
        L.attn_fwd_tile_plan.argtypes = [i, i, i, i, i, vp, vp, vp, vp]
        L.attn_fwd_tile_plan.restype = i
        L.attn_fwd_tile_plan_window.argtypes = [i, i, i, i, i, i, vp, vp, vp, vp]
        L.attn_fwd_tile_plan_window.restype = i
        L.attn_fwd_tile_plan_ex.argtypes = [i, i, i, i, i, i, i, vp, vp, vp, vp]
        L.attn_fwd_tile_plan_ex.restype = i
        L.attn_fwd_trace.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, f, vp, vp, sz,
                                     vp, vp]
        L.attn_fwd_trace.restype = i
        L.attn_device_status.argtypes = [vp, i]
        L.attn_device_status.restype = i
        L.attn_last_device_status.argtypes = [vp]
        L.attn_last_device_status.restype = i
        L.attn_strerror.argtypes = [i]
        L.attn_strerror.restype = ctypes.c_char_p
        L.attn_abi_version.argtypes = []
        L.attn_abi_version.restype = i
        L.attn_fwd_decode_static.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, vp, vp]
        L.attn_fwd_decode_static.restype = i
        L.attn_decode_static_max_bytes.argtypes = []
        L.attn_decode_static_max_bytes.restype = sz
        ll = ctypes.POINTER(ctypes.c_int64)
        L.paged_plan.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp]
        L.paged_plan.restype = i
        L.kv_append.argtypes = [vp, vp, vp, ll, vp, f, i, vp, vp, vp, vp, vp, i, i, i, i, i, i, i,
                                vp]
        L.kv_append.restype = i
        L.attn_fwd_tree.argtypes = [vp, vp, vp, vp, i, i, i, vp, vp, vp, vp, vp, vp, i, i, i, i, i,
                                    i, f, vp, vp, sz, vp]
        L.attn_fwd_tree.restype = i
        L.attn_tree_workspace_size.argtypes = [i, i, i, i, i]
        L.attn_tree_workspace_size.restype = sz
        L.attn_debug_timeout_probe.argtypes = [ctypes.c_ulonglong, vp]
        L.attn_debug_timeout_probe.restype = i
        _lib = L
    return _lib


def _torch():
    import torch
    return torch


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _torch_stream(stream):
    """The torch stream a call is enqueued on (default: the current one)."""
    return _torch().cuda.current_stream() if stream is None else stream


def _stream(stream):
    return ctypes.c_void_p(_torch_stream(stream).cuda_stream)


def _check_tensor(t, name, dtype, ndim=None):
    """Type, dtype, rank and contiguity of one argument (no device check:
    _check_devices does that once every argument is known)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")


def _check_devices(ref, named):
    """Every tensor in `named` ((tensor or None, name) pairs) on ref's CUDA
    device."""
    if not ref.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    for t, n in named:
        if t is not None and t.device != ref.device:
            raise ValueError(f"{n} is on {t.device}, expected {ref.device}")


def _check_io(q, key_lens, out, lse, B, Hq, Nq, extra=()):
    """The arguments every attention wrapper shares: key_lens int32 [B];
    out bf16 with q's shape; lse fp32 [B, Hq, Nq]; all on q's device.
    Shapes are checked before devices, so a mismatch is reported the same way
    on any machine.  A short key_lens or a small out / lse would make the
    kernels read or write past the buffers."""
    torch = _torch()
    if key_lens is not None:
        _check_tensor(key_lens, "key_lens", torch.int32, 1)
        if key_lens.numel() != B:
            raise ValueError(f"key_lens has {key_lens.numel()} entries, expected B = {B}")
    if out is not None:
        _check_tensor(out, "out", torch.bfloat16)
        if tuple(out.shape) != tuple(q.shape):
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {tuple(q.shape)}")
    if lse is not None:
        _check_tensor(lse, "lse", torch.float32)
        if tuple(lse.shape) != (B, Hq, Nq):
            raise ValueError(f"lse has shape {tuple(lse.shape)}, expected {(B, Hq, Nq)}")
    _check_devices(q, [(key_lens, "key_lens"), (out, "out"), (lse, "lse"), *extra])


def _outputs(q, out, lse, return_lse, B, Hq, Nq):
    torch = _torch()
    if out is None:
        out = torch.empty_like(q)
    if return_lse and lse is None:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    return out, lse


def _scratch(nbytes, device, stream):
    """A temporary uint8 workspace for one call on `stream`.  It is allocated
    on the current stream, so it is marked as used by `stream` too: the
    caching allocator then keeps it until `stream` has passed the call."""
    torch = _torch()
    ws = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    s = _torch_stream(stream)
    if s != torch.cuda.current_stream(device):
        ws.record_stream(s)
    return ws


def _raise(rc, what):
    if rc != 0:
        raise AttnError(rc, what)


def _shapes(q, k, v):
    B, Hq, Nq, d = q.shape
    Bk, Hkv, Nk, dk = k.shape
    if tuple(v.shape) != tuple(k.shape) or Bk != B or dk != d:
        raise ValueError(f"shape mismatch q{tuple(q.shape)} k{tuple(k.shape)} v{tuple(v.shape)}")
    return B, Hq, Hkv, Nq, Nk, d


def _qkv(q, k, v, names=("q", "k", "v")):
    torch = _torch()
    for t, n in zip((q, k, v), names):
        _check_tensor(t, n, torch.bfloat16, 4)
    return _shapes(q, k, v)


def attn_fwd(q, k, v, causal=False, scale=None, key_lens=None, out=None, lse=None,
             return_lse=True, stream=None, window=0, align=0):
    """O = softmax(Q K^T * scale + M) V on the GPU.

    q: bf16 [B, Hq, Nq, d]; k, v: bf16 [B, Hkv, Nk, d]; key_lens: int32 [B]
    (device) or None; window: sliding window in keys (0 = none); align: 0
    puts query row i at key position i + Nk - Nq, 1 at i + key_lens[b] - Nq
    (multi-token decode over ragged caches).  Returns (o, lse) (lse fp32
    [B, Hq, Nq], natural log) or o alone when return_lse is False.  Plain
    calls use the library's own workspace; with a window or align = 1 a
    workspace tensor is allocated here and passed to attn_fwd_ex.
    """
    if window or align:
        B, Hq, Hkv, Nq, Nk, d = _qkv(q, k, v)
        _check_devices(q, [(k, "k"), (v, "v")])
        ws = _scratch(attn_workspace_size(B, Hq, Hkv, Nq, Nk, d), q.device, stream)
        return attn_fwd_ws(q, k, v, ws, causal=causal, scale=scale, key_lens=key_lens, out=out,
                           lse=lse, return_lse=return_lse, stream=stream, window=window,
                           align=align)
    B, Hq, Hkv, Nq, Nk, d = _qkv(q, k, v)
    _check_io(q, key_lens, out, lse if return_lse else None, B, Hq, Nq,
              extra=[(k, "k"), (v, "v")])
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out, lse = _outputs(q, out, lse, return_lse, B, Hq, Nq)
    torch = _torch()
    with torch.cuda.device(q.device):
        rc = lib().attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out),
                            _ptr(lse if return_lse else None), B, Hq, Hkv, Nq, Nk, d,
                            int(bool(causal)), float(scale), _ptr(key_lens), _stream(stream))
    _raise(rc, "attn_fwd")
    return (out, lse) if return_lse else out


_registered_ws = {}   # device index -> the tensor registered there (kept alive)


def attn_set_workspace(workspace=None, device=None):
    """Register a caller-owned uint8 CUDA tensor (256-byte aligned) as the
    workspace of attn_fwd on its device, or, with None, go back to the
    library's own workspace on `device` (default: the current device).  The
    tensor is kept referenced here while it is registered."""
    torch = _torch()
    if workspace is None:
        dev = torch.cuda.current_device() if device is None else torch.device(device).index
        with torch.cuda.device(dev):
            rc = lib().attn_set_workspace(None, 0)
        _raise(rc, "attn_set_workspace")
        _registered_ws.pop(dev, None)
        return
    _check_tensor(workspace, "workspace", torch.uint8, 1)
    _check_devices(workspace, [])
    dev = workspace.device.index
    with torch.cuda.device(dev):
        rc = lib().attn_set_workspace(_ptr(workspace), workspace.numel())
    _raise(rc, "attn_set_workspace")
    _registered_ws[dev] = workspace


def attn_workspace_size(B, Hq, Hkv, Nq, Nk, d) -> int:
    return int(lib().attn_workspace_size(B, Hq, Hkv, Nq, Nk, d))


def _check_workspace(workspace):
    if workspace is not None:
        _check_tensor(workspace, "workspace", _torch().uint8, 1)


def attn_fwd_ws(q, k, v, workspace, causal=False, scale=None, key_lens=None, out=None,
                lse=None, return_lse=True, stream=None, window=0, align=0):
    """attn_fwd with a caller-owned workspace (uint8 CUDA tensor); a window or
    align = 1 calls attn_fwd_ex."""
    B, Hq, Hkv, Nq, Nk, d = _qkv(q, k, v)
    _check_workspace(workspace)
    _check_io(q, key_lens, out, lse if return_lse else None, B, Hq, Nq,
              extra=[(k, "k"), (v, "v"), (workspace, "workspace")])
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out, lse = _outputs(q, out, lse, return_lse, B, Hq, Nq)
    ws_bytes = 0 if workspace is None else workspace.numel()
    torch = _torch()
    with torch.cuda.device(q.device):
        if window or align:
            rc = lib().attn_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(out),
                                   _ptr(lse if return_lse else None), B, Hq, Hkv, Nq, Nk, d,
                                   int(bool(causal)), int(window), int(align), float(scale),
                                   _ptr(key_lens), _ptr(workspace), ws_bytes, _stream(stream))
            what = "attn_fwd_ex"
        else:
            rc = lib().attn_fwd_ws(_ptr(q), _ptr(k), _ptr(v), _ptr(out),
                                   _ptr(lse if return_lse else None), B, Hq, Hkv, Nq, Nk, d,
                                   int(bool(causal)), float(scale), _ptr(key_lens),
                                   _ptr(workspace), ws_bytes, _stream(stream))
            what = "attn_fwd_ws"
    _raise(rc, what)
    return (out, lse) if return_lse else out


def attn_fwd_paged(q, k_cache, v_cache, block_table, key_lens, causal=True, scale=None,
                   window=0, workspace=None, out=None, lse=None, return_lse=True, stream=None):
    """Decode over a paged KV cache: q bf16 [B, Hq, Nq, d] (each sequence's
    newest Nq tokens), k_cache/v_cache bf16 [num_pages, Hkv, page_size, d],
    block_table int32 [B, max_pages], key_lens int32 [B] (sequence lengths)."""
    torch = _torch()
    _check_tensor(q, "q", torch.bfloat16, 4)
    _check_tensor(k_cache, "k_cache", torch.bfloat16, 4)
    _check_tensor(v_cache, "v_cache", torch.bfloat16, 4)
    _check_tensor(block_table, "block_table", torch.int32, 2)
    if key_lens is None:
        raise ValueError("attn_fwd_paged needs key_lens (the sequence lengths)")
    _check_workspace(workspace)
    B, Hq, Nq, d = q.shape
    num_pages, Hkv, page_size, dk = k_cache.shape
    if tuple(v_cache.shape) != tuple(k_cache.shape) or dk != d or block_table.shape[0] != B:
        raise ValueError("paged cache shapes do not match q / block_table")
    _check_io(q, key_lens, out, lse if return_lse else None, B, Hq, Nq,
              extra=[(k_cache, "k_cache"), (v_cache, "v_cache"), (block_table, "block_table"),
                     (workspace, "workspace")])
    max_pages = block_table.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out, lse = _outputs(q, out, lse, return_lse, B, Hq, Nq)
    if workspace is None:
        workspace = _scratch(attn_workspace_size(B, Hq, Hkv, Nq, max_pages * page_size, d),
                             q.device, stream)
    ws_bytes = workspace.numel()
    with torch.cuda.device(q.device):
        rc = lib().attn_fwd_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                  max_pages, page_size, num_pages, _ptr(out),
                                  _ptr(lse if return_lse else None), B, Hq, Hkv, Nq, d,
                                  int(bool(causal)), int(window), float(scale), _ptr(key_lens),
                                  _ptr(workspace), ws_bytes, _stream(stream))
    _raise(rc, "attn_fwd_paged")
    return (out, lse) if return_lse else out


def attn_fwd_rope(q, k_rot, v, causal=False, scale=None, key_lens=None, rope_base=10000.0,
                  rope_pairing=0, q_pos_offset=0, workspace=None, out=None, lse=None,
                  return_lse=True, stream=None):
    """Attention with q's RoPE fused in: q un-rotated [B, Hq, Nq, d], k_rot
    keys already rotated (rope_apply), v [B, Hkv, Nk, d].  Row i of every
    sequence is rotated at position q_pos_offset + i."""
    B, Hq, Hkv, Nq, Nk, d = _qkv(q, k_rot, v, ("q", "k_rot", "v"))
    _check_workspace(workspace)
    _check_io(q, key_lens, out, lse if return_lse else None, B, Hq, Nq,
              extra=[(k_rot, "k_rot"), (v, "v"), (workspace, "workspace")])
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out, lse = _outputs(q, out, lse, return_lse, B, Hq, Nq)
    if workspace is None:
        workspace = _scratch(lib().attn_rope_workspace_size(B, Hq, Hkv, Nq, Nk, d), q.device,
                             stream)
    ws_bytes = workspace.numel()
    torch = _torch()
    with torch.cuda.device(q.device):
        rc = lib().attn_fwd_rope(_ptr(q), _ptr(k_rot), _ptr(v), _ptr(out),
                                 _ptr(lse if return_lse else None), B, Hq, Hkv, Nq, Nk, d,
                                 int(bool(causal)), float(scale), _ptr(key_lens),
                                 float(rope_base), int(rope_pairing), int(q_pos_offset),
                                 _ptr(workspace), ws_bytes, _stream(stream))
    _raise(rc, "attn_fwd_rope")
    return (out, lse) if return_lse else out


def attn_fwd_decode_static(q, k, v, scale=None, key_lens=None, out=None, lse=None,
                           return_lse=True, stream=None):
    """Decode (Nq == 1) through the entry point that allocates nothing: its
    scratch is a fixed device array inside the library (see
    attn_fwd_decode_static in include/attn.h).  Same result as attn_fwd."""
    B, Hq, Hkv, Nq, Nk, d = _qkv(q, k, v)
    if Nq != 1:
        raise ValueError("attn_fwd_decode_static takes one query row per sequence (Nq == 1)")
    _check_io(q, key_lens, out, lse if return_lse else None, B, Hq, Nq,
              extra=[(k, "k"), (v, "v")])
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out, lse = _outputs(q, out, lse, return_lse, B, Hq, Nq)
    torch = _torch()
    with torch.cuda.device(q.device):
        rc = lib().attn_fwd_decode_static(_ptr(q), _ptr(k), _ptr(v), _ptr(out),
                                          _ptr(lse if return_lse else None), B, Hq, Hkv, Nk, d,
                                          float(scale), _ptr(key_lens), _stream(stream))
    _raise(rc, "attn_fwd_decode_static")
    return (out, lse) if return_lse else out


def rope_apply(x, base=10000.0, pos_offset=0, pairing=0, out=None, stream=None):
    """RoPE on bf16 [B, H, N, d]; out=x rotates in place."""
    torch = _torch()
    _check_tensor(x, "x", torch.bfloat16, 4)
    if out is not None:
        _check_tensor(out, "out", torch.bfloat16, 4)
        if tuple(out.shape) != tuple(x.shape):
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {tuple(x.shape)}")
    _check_devices(x, [(out, "out")])
    if out is None:
        out = torch.empty_like(x)
    B, H, N, d = x.shape
    with torch.cuda.device(x.device):
        rc = lib().rope_apply(_ptr(x), _ptr(out), B, H, N, d, float(base), int(pos_offset),
                              int(pairing), _stream(stream))
    _raise(rc, "rope_apply")
    return out


# The serving calls run once per step or per layer, often on small tensors,
# where the host is what they cost: they look once at each argument's type,
# device, layout and shape, and for the reason only when one does not fit.

def _same(dev, dtype, *tensors):
    """Whether these are contiguous tensors of dtype on CUDA device `dev`."""
    for t in tensors:
        if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
            return False
    return dev >= 0


def _refuse(ref, args):
    """Raise what is wrong with one of `args` ((tensor, name, dtype, shape)):
    shapes and types of all of them before devices (ref's)."""
    for t, name, dtype, shape in args:
        _check_tensor(t, name, dtype)
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    _check_devices(ref, [(t, name) for t, name, _, _ in args])


class _On:
    """The device and stream of a call.  Makes the device current while the
    call runs.  What is allocated for another stream than the current one comes
    from that stream's memory (a block of the current stream's may still be in
    use by work queued there); what is returned is marked as used by the current
    stream too, so that, once freed, it is kept until that stream has passed."""

    __slots__ = ("guard", "other", "raw", "current")

    def __init__(self, dev, stream):
        torch = _torch()
        self.guard = self.other = self.current = None
        if torch.cuda.current_device() != dev:
            self.guard = torch.cuda.device(dev)
        self.raw = torch._C._cuda_getCurrentRawStream(dev)
        if stream is not None and stream.cuda_stream != self.raw:
            self.other, self.raw = stream, stream.cuda_stream
            self.current = torch.cuda.current_stream(dev)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)
        return False

    def new(self, like, shape, dtype, returned=True):
        if self.other is None:
            return like.new_empty(shape, dtype=dtype)
        with _torch().cuda.stream(self.other):
            t = like.new_empty(shape, dtype=dtype)
        if returned:
            t.record_stream(self.current)
        return t

    def like(self, t):      # of a contiguous tensor
        return _torch().empty_like(t) if self.other is None else self.new(t, t.shape, t.dtype)


def _data(t):
    return None if t is None else t.data_ptr()


def paged_plan(old_lens, new_lens, block_table, free_pages, state, page_size, N, index=None,
               slots=None, state_out=None, stream=None):
    """Pages and cache slots of one step: sequence b goes from old_lens[b] to
    new_lens[b] tokens (int32 [B]).  block_table int32 [B, max_pages] and the
    queue of free pages (free_pages int32 [num_pages], state int32 [2] =
    {head, count}) are updated: growing sequences take pages from the queue's
    head, shrinking ones give theirs back at its tail.  Returns (slots,
    state_out): slots int32 [B, N], the cache slot of the sequence's new token
    i (or index[b, i], int32 [B, N], where given; negative: none), -1 where
    there is none; state_out int32 [2], the queue's new state (a tensor of its
    own: pass it as the next call's state).  Page shortage is reported by
    device_status() (ATTN_ERANGE); the entries that got no page are -1 and are
    passed over when their sequence shrinks."""
    torch = _torch()
    i32 = torch.int32
    try:
        (B, max_pages), (num_pages,) = block_table.shape, free_pages.shape
    except (AttributeError, ValueError):
        _check_tensor(block_table, "block_table", i32, 2)
        _check_tensor(free_pages, "free_pages", i32, 1)
        raise
    args = [(index, "index", i32, (B, N)), (slots, "slots", i32, (B, N)),
            (state_out, "state_out", i32, (2,))]
    args = [x for x in args if x[0] is not None]
    dev = block_table.get_device()
    try:
        ok = (old_lens.shape == new_lens.shape == (B,) and state.shape == (2,)
              and _same(dev, i32, block_table, old_lens, new_lens, free_pages, state)
              and all(t.shape == shape and _same(dev, i32, t) for t, _, _, shape in args))
    except AttributeError:   # not a tensor
        ok = False
    if not ok:
        _refuse(block_table, [(block_table, "block_table", i32, (B, max_pages)),
                              (old_lens, "old_lens", i32, (B,)), (new_lens, "new_lens", i32, (B,)),
                              (free_pages, "free_pages", i32, (num_pages,)),
                              (state, "state", i32, (2,))] + args)
    with _On(dev, stream) as on:
        if slots is None:
            slots = on.new(block_table, (B, N), i32)
        if state_out is None:
            state_out = on.like(state)
        rc = lib().paged_plan(old_lens.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(),
                              free_pages.data_ptr(), state.data_ptr(), state_out.data_ptr(),
                              _data(index), slots.data_ptr(), B, N, max_pages, int(page_size),
                              num_pages, on.raw)
    if rc != 0:
        raise AttnError(rc, "paged_plan")
    return slots, state_out


def _check_rows(t, name, shape):
    """A bf16 [B, H, N, d] argument (of this shape, if one is given) that may
    be a strided view with d contiguous."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.dim() != 4:
        raise ValueError(f"{name} must have 4 dimensions")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.stride(3) != 1 and t.shape[3] > 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")


def kv_append(k, v=None, slots=None, k_cache=None, v_cache=None, q=None, positions=None,
              rope_base=10000.0, rope_pairing=0, return_k=None, q_out=None, k_out=None,
              stream=None):
    """Rotate a step's queries and keys at each token's own position and store
    its keys and values in the cache, in one pass.

    q bf16 [B, Hq, N, d] or None, k and v bf16 [B, Hkv, N, d], strided views
    allowed (d contiguous, other strides multiples of 8 elements); positions
    int32 [B, N] or None (nothing is rotated); slots int32 [B, N] (paged_plan's;
    negative: not stored) with k_cache, v_cache bf16 [num_pages, Hkv,
    page_size, d] (a contiguous cache [B, Hkv, Nk, d] is B pages of Nk rows), or
    None together with v and the caches: nothing is stored.  Slots must be
    distinct.  Returns (q rotated or None, k rotated or None), contiguous; k's
    is made when return_k is set (by default: when nothing is stored) or k_out
    is given.  q_out / k_out may be q / k themselves."""
    torch = _torch()
    bf, i32 = torch.bfloat16, torch.int32
    _check_rows(k, "k", None)
    B, Hkv, N, d = shape = k.shape
    Hq = 0
    rows = [(k, "k")]
    args = []
    if q is not None:
        _check_rows(q, "q", None)
        Bq, Hq, Nq, dq = q.shape
        if Bq != B or Nq != N or dq != d:
            raise ValueError(f"shape mismatch q{tuple(q.shape)} k{tuple(shape)}")
        if positions is None:
            raise ValueError("kv_append rotates q: it needs positions")
        rows.append((q, "q"))
    elif q_out is not None:
        raise ValueError("q_out without q")
    num_pages = page_size = 0
    if slots is not None:
        if v is None or k_cache is None or v_cache is None:
            raise ValueError("v, slots, k_cache and v_cache go together")
        _check_rows(v, "v", shape)
        rows.append((v, "v"))
        _check_tensor(k_cache, "k_cache", bf, 4)
        num_pages, hc, page_size, dc = cs = k_cache.shape
        if hc != Hkv or dc != d:
            raise ValueError(f"cache {tuple(cs)} does not match k{tuple(shape)}")
        args += [(slots, "slots", i32, (B, N)), (k_cache, "k_cache", bf, cs),
                 (v_cache, "v_cache", bf, cs)]
    elif v is not None or k_cache is not None or v_cache is not None:
        raise ValueError("v, slots, k_cache and v_cache go together")
    if positions is not None:
        args.append((positions, "positions", i32, (B, N)))
    if return_k is None:
        return_k = slots is None
    if (return_k or k_out is not None) and positions is None:
        raise ValueError("kv_append returns rotated keys: it needs positions")
    if q_out is not None:
        args.append((q_out, "q_out", bf, q.shape))
    if k_out is not None:
        args.append((k_out, "k_out", bf, shape))
    dev = k.get_device()
    try:
        ok = dev >= 0 and all(t.shape == sh and _same(dev, dt, t) for t, _, dt, sh in args)
    except AttributeError:   # not a tensor
        ok = False
    if not ok:
        _refuse(k, args)
    for t, n in rows:
        if t.get_device() != dev:
            _check_devices(k, [(t, n)])
    kb, kh, kt, _ = k.stride()
    qb, qh, qt, _ = (0, 0, 0, 0) if q is None else q.stride()
    vb, vh, vt, _ = (0, 0, 0, 0) if v is None else v.stride()
    with _On(dev, stream) as on:
        if q is not None and q_out is None:
            q_out = on.new(q, q.shape, bf)
        if return_k and k_out is None:
            k_out = on.new(k, shape, bf)
        rc = lib().kv_append(_data(q), k.data_ptr(), _data(v),
                             _Strides9(qb, qh, qt, kb, kh, kt, vb, vh, vt), _data(positions),
                             rope_base, rope_pairing, _data(q_out), _data(k_out), _data(slots),
                             _data(k_cache), _data(v_cache), B, Hq, Hkv, N, d, page_size,
                             num_pages, on.raw)
    if rc != 0:
        raise AttnError(rc, "kv_append")
    return q_out, k_out


_Strides9 = ctypes.c_int64 * 9


_tree_ws_bytes = {}   # of sizes seen: (device, sizes) -> bytes


def attn_tree_workspace_size(B, Hq, Hkv, Nq, d) -> int:
    return int(lib().attn_tree_workspace_size(B, Hq, Hkv, Nq, d))


def attn_fwd_tree(q, k_cache, v_cache, key_lens, k_new, v_new, parents, new_lens=None,
                  block_table=None, scale=None, workspace=None, out=None, lse=None,
                  return_lse=True, stream=None):
    """Attention for a tree of drafted tokens over a cache: q bf16 [B, Hq, Nq,
    d], the nodes' keys (rotated) and values k_new, v_new bf16 [B, Hkv, Nq,
    d], parents int32 [B, Nq] (the node each one follows, -1: the last cached
    token; parents come first), new_lens int32 [B] nodes per sequence (None:
    Nq).  Every node sees the key_lens[b] cached keys, itself and its
    ancestors.  The cache is paged with a block_table int32 [B, max_pages]
    (k_cache, v_cache bf16 [num_pages, Hkv, page_size, d]), else contiguous
    [B, Hkv, Nk, d] (key_lens None: Nk).  Returns (o, lse) as attn_fwd; rows at
    or beyond new_lens[b] are 0 and -inf."""
    torch = _torch()
    bf, i32 = torch.bfloat16, torch.int32
    try:
        B, Hq, Nq, d = shape = q.shape
        Bn, Hkv, Nn, dn = new = k_new.shape
        _, _, _, _ = cs = k_cache.shape
    except (AttributeError, ValueError):
        for t, n in ((q, "q"), (k_new, "k_new"), (k_cache, "k_cache")):
            _check_tensor(t, n, bf, 4)
        raise
    for t, n in ((v_new, "v_new"), (v_cache, "v_cache")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{n} must be a torch.Tensor")
    if Bn != B or Nn != Nq or dn != d or v_new.shape != new:
        for t, n in ((q, "q"), (k_new, "k_new"), (v_new, "v_new")):
            _check_tensor(t, n, bf, 4)
        raise ValueError(f"shape mismatch q{tuple(shape)} k_new{tuple(new)} "
                         f"v_new{tuple(v_new.shape)}")
    if v_cache.shape != cs or cs[1] != Hkv or cs[3] != d:
        raise ValueError(f"cache shapes {tuple(cs)}, {tuple(v_cache.shape)} do not match "
                         f"k_new{tuple(new)}")
    args = []
    max_pages = num_pages = page_size = Nk = 0
    if block_table is not None:
        if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
            _check_tensor(block_table, "block_table", i32, 2)
        rows, max_pages = block_table.shape
        if rows != B:
            raise ValueError(f"block_table has {rows} rows, expected B = {B}")
        if key_lens is None:
            raise ValueError("attn_fwd_tree over a paged cache needs key_lens")
        args.append((block_table, "block_table", i32, block_table.shape))
        num_pages, page_size = cs[0], cs[2]
    else:
        if cs[0] != B:
            raise ValueError(f"cache has {cs[0]} sequences, expected B = {B}")
        Nk = cs[2]
    if key_lens is not None:
        if not isinstance(key_lens, torch.Tensor) or key_lens.dim() != 1:
            _check_tensor(key_lens, "key_lens", i32, 1)
        if key_lens.numel() != B:
            raise ValueError(f"key_lens has {key_lens.numel()} entries, expected B = {B}")
        args.append((key_lens, "key_lens", i32, (B,)))
    if new_lens is not None:
        args.append((new_lens, "new_lens", i32, (B,)))
    if out is not None:
        args.append((out, "out", bf, shape))
    if not return_lse:
        lse = None
    elif lse is not None:
        args.append((lse, "lse", torch.float32, (B, Hq, Nq)))
    if workspace is not None:
        _check_workspace(workspace)
        args.append((workspace, "workspace", torch.uint8, workspace.shape))
    dev = q.get_device()
    try:
        ok = (_same(dev, bf, q, k_cache, v_cache, k_new, v_new) and parents.shape == (B, Nq)
              and _same(dev, i32, parents)
              and all(t.shape == sh and _same(dev, dt, t) for t, _, dt, sh in args))
    except AttributeError:   # not a tensor
        ok = False
    if not ok:
        _refuse(q, [(q, "q", bf, shape), (k_cache, "k_cache", bf, cs), (v_cache, "v_cache", bf, cs),
                    (k_new, "k_new", bf, new), (v_new, "v_new", bf, new),
                    (parents, "parents", i32, (B, Nq))] + args)
    with _On(dev, stream) as on:
        if out is None:
            out = on.like(q)
        if return_lse and lse is None:
            lse = on.new(q, (B, Hq, Nq), torch.float32)
        L = lib()
        if workspace is None:
            key = (dev, Hq, Hkv, Nq, d, B)
            ws_bytes = _tree_ws_bytes.get(key)
            if ws_bytes is None:
                ws_bytes = _tree_ws_bytes[key] = L.attn_tree_workspace_size(B, Hq, Hkv, Nq, d)
            workspace = on.new(q, (max(ws_bytes, 256),), torch.uint8, returned=False)
        else:
            ws_bytes = workspace.numel()
        rc = L.attn_fwd_tree(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                             _data(block_table), max_pages, page_size, num_pages,
                             k_new.data_ptr(), v_new.data_ptr(), parents.data_ptr(),
                             _data(new_lens), out.data_ptr(), _data(lse), B, Hq, Hkv, Nq, Nk, d,
                             1.0 / math.sqrt(d) if scale is None else scale, _data(key_lens),
                             workspace.data_ptr(), ws_bytes, on.raw)
    if rc != 0:
        raise AttnError(rc, "attn_fwd_tree")
    return (out, lse) if return_lse else out


def prefill_tile_shape(d):
    br, bc = ctypes.c_int(), ctypes.c_int()
    _raise(lib().attn_prefill_tile_shape(d, ctypes.byref(br), ctypes.byref(bc)),
           "attn_prefill_tile_shape")
    return br.value, bc.value


def tile_plan(B, Nq, Nk, d, causal, key_lens=None, device="cuda", stream=None, window=0,
              align=0):
    """(first, count) int32 [B, nqt] tensors: the KV tiles the prefill kernel
    visits for each (b, query tile), optionally under a sliding window."""
    torch = _torch()
    br, _ = prefill_tile_shape(d)
    nqt = -(-Nq // br)
    first = torch.empty((B, nqt), dtype=torch.int32, device=device)
    count = torch.empty((B, nqt), dtype=torch.int32, device=device)
    rc = lib().attn_fwd_tile_plan_ex(B, Nq, Nk, d, int(bool(causal)), int(window), int(align),
                                     _ptr(key_lens), _ptr(first), _ptr(count), _stream(stream))
    _raise(rc, "attn_fwd_tile_plan_ex")
    return first, count


def prefill_trace(q, k, v, causal=False, scale=None, key_lens=None, window=0, align=0,
                  stream=None):
    """Run the prefill kernel with its trace hook: returns (o, lse, trace),
    trace int32 [B, Hq, nqt, 3] = {first, last, count} of the KV tiles whose
    scores the kernel computed for each query tile ({-1, -1, 0} for none)."""
    B, Hq, Hkv, Nq, Nk, d = _qkv(q, k, v)
    _check_io(q, key_lens, None, None, B, Hq, Nq, extra=[(k, "k"), (v, "v")])
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    torch = _torch()
    br, _ = prefill_tile_shape(d)
    nqt = -(-Nq // br)
    trace = torch.tensor([-1, -1, 0], dtype=torch.int32, device=q.device).repeat(B * Hq * nqt)
    out, lse = _outputs(q, None, None, True, B, Hq, Nq)
    ws = _scratch(attn_workspace_size(B, Hq, Hkv, Nq, Nk, d), q.device, stream)
    with torch.cuda.device(q.device):
        rc = lib().attn_fwd_trace(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv,
                                  Nq, Nk, d, int(bool(causal)), int(window), int(align),
                                  float(scale), _ptr(key_lens), _ptr(ws), ws.numel(),
                                  _ptr(trace), _stream(stream))
    _raise(rc, "attn_fwd_trace")
    return out, lse, trace.view(B, Hq, nqt, 3)


def device_status(reset=True, stream=None) -> int:
    """Synchronise and read the library's device status word (0 = OK)."""
    return int(lib().attn_device_status(_stream(stream), int(bool(reset))))


def attn_last_device_status(stream=None) -> int:
    """Synchronise, return the status since the last read and clear it."""
    return int(lib().attn_last_device_status(_stream(stream)))
