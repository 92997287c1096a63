"""Python binding of libkpool (ctypes).  Argument marshalling only.

Every step of the selection runs in the HIP library; this module passes
torch tensors' device pointers and the current HIP stream through the C ABI
declared in include/kpool.h, allocates outputs with torch (device memory is
all torch is used for) and turns negative status codes into exceptions.
There is no CPU fallback: if libkpool.so is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkpool.so")

KPOOL_OK, KPOOL_EINVAL, KPOOL_EUNSUPPORTED, KPOOL_EWORKSPACE, KPOOL_EHIP = 0, -1, -2, -3, -4
KPOOL_FLAG_OVERLAP = 1
KPOOL_FLAG_TAIL = 2
PROFILE_KINDS = ("pool_keys", "score", "topk", "expand", "scores_copy")
LAYER_PROFILE_KINDS = ("norm", "attend")
KPOOL_DTYPE_BF16, KPOOL_DTYPE_F32 = 0, 1
KPOOL_ROTARY_INTERLEAVED, KPOOL_ROTARY_INVERSE = 1, 2

_lib = None


class KpoolError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn} failed with status {status}: {msg}")
        self.status = status


def lib():
    """The loaded libkpool.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libkpool.so is not built ({LIB_PATH}); run __graft_entry__.build()")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    u32 = ctypes.c_uint32
    sig = {
        "kpool_last_error": (ctypes.c_char_p, []),
        "kpool_version": (ctypes.c_int, []),
        "kpool_count_pools": (i64, [vp, i32, i32, u32, vp, vp]),
        "kpool_pool_keys": (ctypes.c_int, [vp, vp, vp, vp, i32, i32, i32, u32, vp, vp]),
        "kpool_pool_keys_gated": (ctypes.c_int, [vp, vp, vp, vp, vp, vp, i32, i32, i32, u32, vp, vp]),
        "kpool_workspace_bytes": (sz, [i64, i64, i32, i32]),
        "kpool_chunk_rows": (i64, [i32, sz, u32, vp]),
        "kpool_score_topk": (ctypes.c_int, [vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, i64, i64,
                                            i32, vp, sz, u32, vp, vp, vp]),
        "kpool_score_topk_noalloc": (ctypes.c_int, [vp, vp, vp, vp, vp, i32, i32, i32, i32, f32,
                                                    i64, i64, i32, u32, vp, vp, vp]),
        "kpool_expand": (ctypes.c_int, [vp, vp, vp, i32, i32, i64, i64, i32, u32, vp, vp]),
        "kpool_topk": (ctypes.c_int, [vp, i64, vp, i64, i32, vp, vp]),
        "kpool_attend_workspace_bytes": (sz, [vp, vp, i32, i32, i32, i32]),
        "kpool_attend": (ctypes.c_int, [vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, i32, i32, i32, i32,
                                        f32, vp, sz, vp, vp, vp]),
        "kpool_attend_backward_workspace_bytes": (sz, [vp, vp, i32, i32, i32, i32]),
        "kpool_attend_backward": (ctypes.c_int, [vp, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, vp, vp,
                                                 i32, i32, i32, i32, f32, vp, sz, vp, vp, vp, vp]),
        "kpool_attend_selected_workspace_bytes": (sz, [i64, i32, i32, i32, i32, i32]),
        "kpool_attend_selected": (ctypes.c_int, [vp, i64, vp, i64, vp, i64, vp, i32, vp, vp, vp, vp, i32,
                                                 i32, i32, i32, f32, vp, sz, vp, vp, vp]),
        "kpool_layer_norm": (ctypes.c_int, [vp, i64, vp, vp, i64, i32, f32, i32, vp, vp, vp, vp]),
        "kpool_layer_norm_backward_workspace_bytes": (sz, [i64, i32]),
        "kpool_layer_norm_backward": (ctypes.c_int, [vp, vp, i64, vp, vp, vp, i64, i32, i32, vp, sz,
                                                     vp, vp, vp, vp]),
        "kpool_attend_expanded_workspace_bytes": (sz, [vp, vp, i32, i32, i32, i32, i32]),
        "kpool_attend_expanded": (ctypes.c_int, [vp, i64, vp, i64, i64, vp, i64, vp, i64, i64, vp, vp, vp, vp, i32, i32,
                                                 i32, i32, i32, f32, vp, sz, vp, vp, vp]),
        "kpool_attend_expanded_backward_workspace_bytes": (sz, [vp, vp, i32, i32, i32, i32, i32]),
        "kpool_attend_expanded_backward": (ctypes.c_int, [vp, vp, i64, vp, i64, i64, vp, i64, vp, i64, i64, vp, vp, vp, vp,
                                                          vp, vp, i32, i32, i32, i32, i32, f32, vp, sz, vp, vp, vp, vp, vp]),
        "kpool_attend_latent_workspace_bytes": (sz, [vp, i32, i32, i32, i32, i32]),
        "kpool_attend_latent": (ctypes.c_int, [vp, i64, vp, i64, i64, vp, i32, i32, vp, vp, i32, vp, vp, i32, i32, i32,
                                               i32, f32, vp, sz, vp, vp, vp]),
        "kpool_attend_latent_selected_workspace_bytes": (sz, [i64, i32, i32, i32, i32]),
        "kpool_attend_latent_selected": (ctypes.c_int, [vp, i64, vp, i64, i64, vp, i32, i32, vp, vp, vp, i32, vp, vp, i32,
                                                        i32, i32, i32, f32, vp, sz, vp, vp, vp]),
        "kpool_rotary": (ctypes.c_int, [vp, i64, vp, vp, i64, i32, i32, i32, i32, f32, i32, u32, vp, i64, vp]),
        "kpool_profile_enable": (ctypes.c_int, [ctypes.c_int]),
        "kpool_profile_collect": (ctypes.c_int, [vp, vp]),
        "kpool_layer_profile_collect": (ctypes.c_int, [vp, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def _check(rc, fn):
    if rc != KPOOL_OK:
        raise KpoolError(fn, int(rc), lib().kpool_last_error().decode())


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _host_i32(a):
    a = np.ascontiguousarray(np.asarray(a, dtype=np.int32))
    return a, a.ctypes.data_as(ctypes.c_void_p)


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _on(stream):
    """Context in which the wrappers allocate: the stream the library call will run on.

    torch's caching allocator hands a freed block out again only to work ordered
    after the frees on the block's own stream; allocating on the call's stream
    keeps a workspace or output from being reused while the call still uses it."""
    import contextlib

    import torch
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _need(t, name, elem_size=None, dtype=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous device tensor")
    if elem_size is not None and t.element_size() != elem_size:
        raise ValueError(f"{name} must have {elem_size}-byte elements")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")


# ---------------------------------------------------------------------------
# The C ABI, one wrapper per entry point
# ---------------------------------------------------------------------------

def version() -> int:
    return lib().kpool_version()


def _tail(tail):
    return KPOOL_FLAG_TAIL if tail else 0


def count_pools(cu_seqlens, kpool: int, tail: bool = False):
    """(cu_pools int32 [nseq+1], max_pools, P_tot) for a host cu_seqlens (tail: full pools)."""
    cu, cup = _host_i32(cu_seqlens)
    nseq = len(cu) - 1
    out = np.zeros(max(nseq, 0) + 1, dtype=np.int32)
    mx = ctypes.c_int32(0)
    tot = lib().kpool_count_pools(cup, nseq, kpool, _tail(tail), out.ctypes.data_as(ctypes.c_void_p),
                                  ctypes.byref(mx))
    _check(0 if tot >= 0 else tot, "kpool_count_pools")
    return out, int(mx.value), int(tot)


def workspace_bytes(q_lo: int, q_hi: int, max_pools: int, nbuf: int = 2) -> int:
    """Workspace of score_topk over rows [q_lo, q_hi): nbuf chunk buffers (2 for the
    chunk overlap, 1 without), each capped at 2 GiB of fp32 scores."""
    return int(lib().kpool_workspace_bytes(q_lo, q_hi, max_pools, nbuf))


def chunk_rows(max_pools: int, workspace_bytes: int, overlap: bool = False, tail: bool = False):
    """(rows per chunk, chunk buffers) of score_topk's chunk loop for this workspace."""
    nbuf = ctypes.c_int32(0)
    rows = lib().kpool_chunk_rows(max_pools, workspace_bytes,
                                  (KPOOL_FLAG_OVERLAP if overlap else 0) | _tail(tail), ctypes.byref(nbuf))
    _check(0 if rows >= 0 else rows, "kpool_chunk_rows")
    return int(rows), int(nbuf.value)


def pool_keys(k, cu_seqlens, cu_seqlens_dev, cu_pools_dev, kpool: int, out=None, stream=None,
              tail: bool = False):
    import torch
    _need(k, "k", 2)
    cu, cup = _host_i32(cu_seqlens)
    nseq = len(cu) - 1
    _, _, P_tot = count_pools(cu, kpool, tail)
    D = k.shape[-1]
    if out is None:
        with _on(stream):
            out = torch.empty((P_tot, D), dtype=k.dtype, device=k.device)
    rc = lib().kpool_pool_keys(_p(k), cup, _p(cu_seqlens_dev), _p(cu_pools_dev), nseq, D, kpool,
                               _tail(tail), _p(out), _stream(stream))
    _check(rc, "kpool_pool_keys")
    return out


def pool_keys_gated(k, g, ape, cu_seqlens, cu_seqlens_dev, cu_pools_dev, kpool: int, out=None,
                    stream=None, tail: bool = False):
    """Gated pooled keys: k, g bf16 [T, D] (int16 storage), ape fp32 [kpool, D]."""
    import torch
    _need(k, "k", 2)
    _need(g, "g", 2)
    _need(ape, "ape", dtype=torch.float32)
    cu, cup = _host_i32(cu_seqlens)
    nseq = len(cu) - 1
    _, _, P_tot = count_pools(cu, kpool, tail)
    D = k.shape[-1]
    if tuple(g.shape) != tuple(k.shape) or tuple(ape.shape) != (kpool, D):
        raise ValueError("need g shaped like k and ape [kpool, D]")
    if out is None:
        with _on(stream):
            out = torch.empty((P_tot, D), dtype=k.dtype, device=k.device)
    rc = lib().kpool_pool_keys_gated(_p(k), _p(g), _p(ape), cup, _p(cu_seqlens_dev), _p(cu_pools_dev),
                                     nseq, D, kpool, _tail(tail), _p(out), _stream(stream))
    _check(rc, "kpool_pool_keys_gated")
    return out


def score_topk(q, kp, w, cu_seqlens, cu_seqlens_dev, kpool: int, budget: int, q_lo: int = 0,
               q_hi: int | None = None, scale: float | None = None, workspace=None,
               pool_ids=None, scores_out=None, want_scores: bool = False, overlap: bool = False,
               stream=None, tail: bool = False):
    """Run the chunked score + top-k for rows [q_lo, q_hi).  Returns (pool_ids, scores_out).

    overlap=True passes KPOOL_FLAG_OVERLAP (two chunk buffers on two streams); a
    workspace allocated here then holds two chunk buffers, otherwise one."""
    return _score_topk(q, 0, kp, w, cu_seqlens, cu_seqlens_dev, kpool, budget, q_lo, q_hi, scale, workspace, pool_ids,
                       scores_out, want_scores, overlap, stream, tail)


def _score_topk(q, first, kp, w, cu_seqlens, cu_seqlens_dev, kpool, budget, q_lo, q_hi, scale, workspace, pool_ids,
                scores_out, want_scores, overlap, stream, tail):
    """score_topk where q holds the batch's rows from `first` <= q_lo on (the library reads the rows [q_lo, q_hi) alone)."""
    import torch
    _need(q, "q", 2)
    _need(kp, "kp", 2)
    _need(w, "w", dtype=torch.float32)
    cu, cup = _host_i32(cu_seqlens)
    nseq = len(cu) - 1
    T = int(cu[-1])
    if q_hi is None:
        q_hi = T
    H, D = q.shape[-2], q.shape[-1]
    if scale is None:
        scale = float(np.float32(1.0) / np.sqrt(np.float32(D)))
    _, max_pools, _ = count_pools(cu, kpool, tail)
    rows = max(0, q_hi - q_lo)
    with _on(stream):
        if pool_ids is None:
            pool_ids = torch.empty((rows, budget), dtype=torch.int32, device=q.device)
        if want_scores and scores_out is None:
            scores_out = torch.empty((rows, max_pools), dtype=torch.float32, device=q.device)
        if workspace is None:
            nb = workspace_bytes(q_lo, q_hi, max_pools, 2 if overlap else 1)
            workspace = torch.empty(max(nb, 16), dtype=torch.uint8, device=q.device)
    q_at = q.data_ptr() - first * H * D * q.element_size()  # (where row 0 would be)
    rc = lib().kpool_score_topk(ctypes.c_void_p(q_at), _p(kp), _p(w), cup, _p(cu_seqlens_dev), nseq, H, D, kpool,
                                ctypes.c_float(scale), q_lo, q_hi, budget, _p(workspace),
                                workspace.numel() * workspace.element_size(),
                                (KPOOL_FLAG_OVERLAP if overlap else 0) | _tail(tail), _p(pool_ids),
                                _p(scores_out), _stream(stream))
    _check(rc, "kpool_score_topk")
    return pool_ids, scores_out


def score_topk_noalloc(q, kp, w, cu_seqlens, cu_seqlens_dev, kpool: int, budget: int,
                       q_lo: int, q_hi: int, pool_ids, scores_out=None, scale: float | None = None,
                       stream=None, tail: bool = False):
    """score_topk through the library's static scratch (kpool_score_topk_noalloc): the
    caller passes every output; nothing is allocated here or in the library."""
    import torch
    _need(q, "q", 2)
    _need(kp, "kp", 2)
    _need(w, "w", dtype=torch.float32)
    cu, cup = _host_i32(cu_seqlens)
    H, D = q.shape[-2], q.shape[-1]
    if scale is None:
        scale = float(np.float32(1.0) / np.sqrt(np.float32(D)))
    rc = lib().kpool_score_topk_noalloc(_p(q), _p(kp), _p(w), cup, _p(cu_seqlens_dev), len(cu) - 1,
                                        H, D, kpool, ctypes.c_float(scale), q_lo, q_hi, budget,
                                        _tail(tail), _p(pool_ids), _p(scores_out), _stream(stream))
    _check(rc, "kpool_score_topk_noalloc")
    return pool_ids, scores_out


def expand(pool_ids, cu_seqlens, cu_seqlens_dev, kpool: int, budget: int, q_lo: int = 0,
           q_hi: int | None = None, out=None, stream=None, tail: bool = False):
    """Token ids [rows, budget*kpool] (+ kpool - 1 tail slots in tail mode)."""
    import torch
    cu, cup = _host_i32(cu_seqlens)
    nseq = len(cu) - 1
    if q_hi is None:
        q_hi = int(cu[-1])
    rows = max(0, q_hi - q_lo)
    if out is None:
        with _on(stream):
            out = torch.empty((rows, budget * kpool + (kpool - 1 if tail else 0)), dtype=torch.int32,
                              device=pool_ids.device)
    rc = lib().kpool_expand(_p(pool_ids), cup, _p(cu_seqlens_dev), nseq, kpool, q_lo, q_hi, budget,
                            _tail(tail), _p(out), _stream(stream))
    _check(rc, "kpool_expand")
    return out


def topk(scores, n_valid, budget: int, out=None, stream=None):
    """Selection alone over fp32 scores [rows, ld] with n_valid int32 [rows] (device)."""
    import torch
    _need(scores, "scores", dtype=torch.float32)
    rows, ld = scores.shape
    if out is None:
        with _on(stream):
            out = torch.empty((rows, budget), dtype=torch.int32, device=scores.device)
    rc = lib().kpool_topk(_p(scores), ld, _p(n_valid), rows, budget, _p(out), _stream(stream))
    _check(rc, "kpool_topk")
    return out


class _OnDevice:
    """The call's stream (by default the current one of t's device) made current along with
    t's device, so that outputs and workspaces allocated inside belong to that stream; gives
    its handle."""

    __slots__ = ("handle", "contexts")

    def __init__(self, t, stream):
        import torch
        index = t.get_device()
        if stream is None and torch._C._cuda_getDevice() == index:  # (t has initialised HIP)
            self.contexts = None
            self.handle = torch._C._cuda_getCurrentRawStream(index)
            return
        if stream is not None and stream.device != t.device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
        self.contexts = [torch.cuda.device(index)]
        if stream is not None:
            self.contexts.append(torch.cuda.stream(stream))

    def __enter__(self):
        if self.contexts is None:
            return self.handle
        import torch
        for c in self.contexts:
            c.__enter__()
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())

    def __exit__(self, *exc):
        if self.contexts is not None:
            for c in reversed(self.contexts):
                c.__exit__(*exc)


def _host_address(a):
    """A host array's address (the quick way needs a writable one)."""
    try:
        return ctypes.addressof(ctypes.c_char.from_buffer(a))
    except TypeError:
        return a.__array_interface__["data"][0]


def _at(t):
    """A tensor's address for a call (None for none)."""
    return None if t is None else t.data_ptr()


def _like(t, name, shape, dtype, device):
    """An output or parameter given by the caller: contiguous, of this shape, type and device."""
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(shape)} on {device}")


def _int32(**numbers):
    """Numbers for 32-bit arguments, of which ctypes would pass the low bits alone."""
    for name, x in numbers.items():
        if not -2 ** 31 <= x < 2 ** 31:
            raise ValueError(f"{name} must fit 32 bits (got {x})")


def _refuse_graph(fn, *tensors):
    """Results are plain tensors: where autograd would record the call, its gradients would be lost
    without a word."""
    import torch
    if any(t is not None and t.requires_grad for t in tensors) and torch.is_grad_enabled():
        raise ValueError(f"{fn} records no autograd graph: call it under torch.no_grad() or from the forward of a "
                         f"torch.autograd.Function, on detached tensors otherwise")


def _heads(t, name, device, codes):
    """t as packed tokens [T, H, D] of bf16 with any token stride: (T, H, D, stride)."""
    if t.dim() != 3 or not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a device tensor [T, heads, D] on {device}")
    if t.dtype not in codes:
        raise ValueError(f"{name} must be bfloat16 (or int16 bit patterns)")
    T, H, D = t.shape
    s0, s1, s2 = t.stride()
    if (s2 != 1 and D > 1) or (s1 != D and H > 1):
        raise ValueError(f"the heads of a token of {name} must be contiguous")
    return T, H, D, s0 if T > 1 else H * D


def _cu_pair(cu_q, cu_q_dev, cu_k, cu_k_dev, device):
    """Host arrays and device copies of both lengths; no keys' lengths given: the queries'."""
    import torch
    if (cu_k is None) != (cu_k_dev is None):
        raise ValueError("give both cu_k and cu_k_dev, or neither")
    cu_q = np.ascontiguousarray(cu_q, dtype=np.int32)
    cu_k = cu_q if cu_k is None else np.ascontiguousarray(cu_k, dtype=np.int32)
    if cu_q.ndim != 1 or len(cu_q) < 2 or cu_k.shape != cu_q.shape:
        raise ValueError("cu_q and cu_k must be 1-dimensional with nseq + 1 entries each")
    _like(cu_q_dev, "cu_q_dev", cu_q.shape, torch.int32, device)
    if cu_k_dev is None:
        cu_k_dev = cu_q_dev
    else:
        _like(cu_k_dev, "cu_k_dev", cu_q.shape, torch.int32, device)
    return cu_q, cu_q_dev, cu_k, cu_k_dev


class _Attend:
    """The arguments that the attention calls share, checked."""

    def __init__(self, q, k, v, cu_q, cu_q_dev, cu_k, cu_k_dev, scale):
        import torch
        codes = (torch.bfloat16, torch.int16)
        self.device = device = q.device
        tq, self.Hq, self.D, qs = _heads(q, "q", device, codes)
        tk, self.Hkv, d, ks = _heads(k, "k", device, codes)
        tv, hv, dv, vs = _heads(v, "v", device, codes)
        if hv != self.Hkv or dv != d or d != self.D:
            raise ValueError("q, k and v must agree in D, and k and v in their heads")
        self.cu_q, q_dev, self.cu_k, k_dev = _cu_pair(cu_q, cu_q_dev, cu_k, cu_k_dev, device)
        q_ptr = _host_address(self.cu_q)
        k_ptr = q_ptr if self.cu_k is self.cu_q else _host_address(self.cu_k)
        self.nseq = len(self.cu_q) - 1
        self.Tq, self.Tk = int(self.cu_q[-1]), int(self.cu_k[-1])
        if tq < self.Tq or min(tk, tv) < self.Tk:
            raise ValueError("q, k or v has fewer tokens than its cumulative lengths say")
        self.scale = float(np.float32(1.0) / np.sqrt(np.float32(self.D))) if scale is None else scale
        self.lens = (q_ptr, k_ptr, self.nseq, self.Hq, self.Hkv, self.D)
        self.rows = (q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs)
        self.cu = (q_ptr, q_dev.data_ptr(), k_ptr, k_dev.data_ptr(), self.nseq, self.Hq, self.Hkv, self.D, self.scale)

    def outputs(self, q, out, lse, want_lse):
        import torch
        if out is None:
            rows, width = self.Hq * self.D, self.D
            out = torch.empty_strided((self.Tq, self.Hq, width), (rows, width, 1), dtype=q.dtype, device=self.device)
        else:
            _like(out, "out", (self.Tq, self.Hq, self.D), q.dtype, self.device)
        if lse is not None:
            _like(lse, "lse", (self.Tq, self.Hq), torch.float32, self.device)
        elif want_lse:
            lse = torch.empty_strided((self.Tq, self.Hq), (self.Hq, 1), dtype=torch.float32, device=self.device)
        return out, lse

    def scratch(self, workspace, nbytes):
        import torch
        if workspace is None and nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        return workspace


def _attend_bytes(fn, cu_q, cu_k, Hq, Hkv, D):
    cu_q, qp = _host_i32(cu_q)
    cu_k, kp = _host_i32(cu_k)
    if cu_q.ndim != 1 or cu_k.shape != cu_q.shape:
        raise ValueError("cu_q and cu_k must be 1-dimensional with nseq + 1 entries each")
    nb = int(getattr(lib(), fn)(qp, kp, len(cu_q) - 1, Hq, Hkv, D))
    msg = lib().kpool_last_error().decode()
    if msg:
        raise KpoolError(fn, KPOOL_EINVAL, msg)
    return nb


def attend_workspace_bytes(cu_q, cu_k, Hq: int, Hkv: int, D: int) -> int:
    """Workspace of attend for these sequences (0 where it needs none)."""
    return _attend_bytes("kpool_attend_workspace_bytes", cu_q, cu_k, Hq, Hkv, D)


def attend(q, k, v, cu_q, cu_q_dev, cu_k=None, cu_k_dev=None, scale: float | None = None, out=None,
           want_lse: bool = False, lse=None, workspace=None, stream=None):
    """Causal attention of packed query rows over all the keys they see: (o, lse or None).

    q bf16 [Tq, Hq, D], k and v bf16 [Tk, Hkv, D] (any token stride; each key head serves
    Hq / Hkv query heads); cu_q, cu_k host arrays of nseq + 1 cumulative lengths and their
    device copies, the keys' being the queries' where they are left out.  A sequence's queries
    are the last rows of its keys.  scale is 1 / sqrt(D) by default.  Autograd does not record the
    call (tensors that require gradients are refused where it would); attend_backward has its
    gradients."""
    _refuse_graph("attend", q, k, v)
    a = _Attend(q, k, v, cu_q, cu_q_dev, cu_k, cu_k_dev, scale)
    with _OnDevice(q, stream) as s:
        out, lse = a.outputs(q, out, lse, want_lse)
        ws = a.scratch(workspace, int(lib().kpool_attend_workspace_bytes(*a.lens)))
        rc = lib().kpool_attend(*a.rows, *a.cu, _at(ws), _bytes(ws, q.device), _at(out), _at(lse), s)
    _check(rc, "kpool_attend")
    return out, lse


def attend_backward_workspace_bytes(cu_q, cu_k, Hq: int, Hkv: int, D: int) -> int:
    """Workspace of attend_backward for these sequences."""
    return _attend_bytes("kpool_attend_backward_workspace_bytes", cu_q, cu_k, Hq, Hkv, D)


def attend_backward(d_o, q, k, v, o, lse, cu_q, cu_q_dev, cu_k=None, cu_k_dev=None,
                    scale: float | None = None, workspace=None, dq=None, dk=None, dv=None, stream=None):
    """Gradients (dq, dk, dv) of attend: d_o is the gradient of o [Tq, Hq, D]; o and lse are what
    attend returned (want_lse=True); the rest are its arguments.  dq is [Tq, Hq, D], dk and dv
    [Tk, Hkv, D], in bf16."""
    import torch
    a = _Attend(q, k, v, cu_q, cu_q_dev, cu_k, cu_k_dev, scale)
    rows = (a.Tq, a.Hq, a.D)
    _like(d_o, "d_o", rows, q.dtype, q.device)
    _like(o, "o", rows, q.dtype, q.device)
    _like(lse, "lse", rows[:2], torch.float32, q.device)
    with _OnDevice(q, stream) as s:
        out = []
        for t, name, shape in ((dq, "dq", rows), (dk, "dk", (a.Tk, a.Hkv, a.D)), (dv, "dv", (a.Tk, a.Hkv, a.D))):
            if t is None:
                t = torch.empty(shape, dtype=q.dtype, device=q.device)
            else:
                _like(t, name, shape, q.dtype, q.device)
            out.append(t)
        ws = a.scratch(workspace, int(lib().kpool_attend_backward_workspace_bytes(*a.lens)))
        rc = lib().kpool_attend_backward(_at(d_o), *a.rows, _at(o), _at(lse), *a.cu, _at(ws),
                                         _bytes(ws, q.device), *(_at(t) for t in out), s)
    _check(rc, "kpool_attend_backward")
    return tuple(out)


def attend_selected_workspace_bytes(Tq: int, nseq: int, width: int, Hq: int, Hkv: int, D: int) -> int:
    """Workspace of attend_selected for these sizes (0 where it needs none)."""
    nb = int(lib().kpool_attend_selected_workspace_bytes(Tq, nseq, width, Hq, Hkv, D))
    msg = lib().kpool_last_error().decode()
    if msg:
        raise KpoolError("kpool_attend_selected_workspace_bytes", KPOOL_EINVAL, msg)
    return nb


def attend_selected(q, k, v, token_ids, cu_q, cu_q_dev, cu_k=None, cu_k_dev=None,
                    scale: float | None = None, out=None, want_lse: bool = False, lse=None,
                    workspace=None, stream=None):
    """Attention of packed query rows over the tokens each selected: (o, lse or None).

    token_ids int32 [Tq, width]: sequence-local token ids as expand gives them; entries that
    are negative or past the row stand for nothing.  The rest is attend's, but for a backward
    pass, which there is none of."""
    import torch
    _refuse_graph("attend_selected", q, k, v)
    a = _Attend(q, k, v, cu_q, cu_q_dev, cu_k, cu_k_dev, scale)
    if token_ids.dim() != 2:
        raise ValueError("token_ids must be [Tq, width]")
    width = token_ids.shape[1]
    _like(token_ids, "token_ids", (a.Tq, width), torch.int32, q.device)
    with _OnDevice(q, stream) as s:
        out, lse = a.outputs(q, out, lse, want_lse)
        ws = a.scratch(workspace, int(lib().kpool_attend_selected_workspace_bytes(
            a.Tq, a.nseq, width, a.Hq, a.Hkv, a.D)))
        rc = lib().kpool_attend_selected(*a.rows, _at(token_ids), width, *a.cu, _at(ws),
                                         _bytes(ws, q.device), _at(out), _at(lse), s)
    _check(rc, "kpool_attend_selected")
    return out, lse


def _spaced_heads(t, name, device, codes):
    """t as packed tokens [T, H, D] of bf16: (T, H, D, stride, head stride); the library takes strides whose heads
    lie within their token's."""
    if t.dim() != 3 or not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a device tensor [T, heads, D] on {device}")
    if t.dtype not in codes:
        raise ValueError(f"{name} must be bfloat16 (or int16 bit patterns)")
    T, H, D = t.shape
    s0, s1, s2 = t.stride()
    if s2 != 1 and D > 1:
        raise ValueError(f"the values of a head of {name} must be contiguous")
    s1 = s1 if H > 1 else D
    return T, H, D, s0 if T > 1 else (H - 1) * s1 + D, s1


class _Expanded:
    """The arguments that the expanded form's calls share, checked."""

    def __init__(self, q, k, k_pe, v, cu_q, cu_q_dev, cu_k, cu_k_dev, scale):
        import torch
        codes = (torch.bfloat16, torch.int16)
        self.device = device = q.device
        tq, self.Hq, width, qs = _heads(q, "q", device, codes)
        tk, self.Hkv, self.D, ks, kh = _spaced_heads(k, "k", device, codes)
        tv, hv, dv, vs, vh = _spaced_heads(v, "v", device, codes)
        if k_pe.dim() != 2:
            raise ValueError("k_pe must be [T, P]")
        tp, _, self.P, ps, _ = _spaced_heads(k_pe[:, None], "k_pe", device, codes)
        if hv != self.Hkv or dv != self.D or width != self.D + self.P:
            raise ValueError("k and v must agree in their heads and D, and q have D + P values a head")
        self.cu_q, q_dev, self.cu_k, k_dev = _cu_pair(cu_q, cu_q_dev, cu_k, cu_k_dev, device)
        q_ptr = _host_address(self.cu_q)
        k_ptr = q_ptr if self.cu_k is self.cu_q else _host_address(self.cu_k)
        self.Tq, self.Tk = int(self.cu_q[-1]), int(self.cu_k[-1])
        if tq < self.Tq or min(tk, tv, tp) < self.Tk:
            raise ValueError("q, k, k_pe or v has fewer tokens than its cumulative lengths say")
        nseq = len(self.cu_q) - 1
        scale = float(np.float32(1.0) / np.sqrt(np.float32(width))) if scale is None else scale
        self.lens = (q_ptr, k_ptr, nseq, self.Hq, self.Hkv, self.D, self.P)
        self.rows = (q.data_ptr(), qs, k.data_ptr(), ks, kh, k_pe.data_ptr(), ps, v.data_ptr(), vs, vh)
        self.cu = (q_ptr, q_dev.data_ptr(), k_ptr, k_dev.data_ptr(), nseq, self.Hq, self.Hkv, self.D, self.P, scale)


def _expanded_bytes(fn, cu_q, cu_k, Hq, Hkv, D, P):
    _int32(Hq=Hq, Hkv=Hkv, D=D, P=P)
    cu_q, qp = _host_i32(cu_q)
    cu_k, kp = _host_i32(cu_k)
    if cu_q.ndim != 1 or cu_k.shape != cu_q.shape:
        raise ValueError("cu_q and cu_k must be 1-dimensional with nseq + 1 entries each")
    return _latent_bytes(fn, qp, kp, len(cu_q) - 1, Hq, Hkv, D, P)


def attend_expanded_workspace_bytes(cu_q, cu_k, Hq: int, Hkv: int, D: int, P: int) -> int:
    """Workspace of attend_expanded for these sequences (0 where it needs none)."""
    return _expanded_bytes("kpool_attend_expanded_workspace_bytes", cu_q, cu_k, Hq, Hkv, D, P)


def attend_expanded(q, k, k_pe, v, cu_q, cu_q_dev, cu_k=None, cu_k_dev=None, scale: float | None = None, out=None,
                    want_lse: bool = False, lse=None, workspace=None, stream=None):
    """Latent attention with expanded keys and values, as attend: (o, lse or None).

    q bf16 [Tq, Hq, D + P]; k and v bf16 [Tk, Hkv, D], a token's heads side by side (the two halves of one
    projection's heads, say; keys stored head by head are refused); k_pe bf16 [Tk, P], the keys' positional
    part, which all heads share; strides are multiples of 8.  scale is 1 / sqrt(D + P) by default; the rest is attend's.  attend_expanded_backward has its gradients; new
    tokens over a cache take attend_latent."""
    import torch
    _refuse_graph("attend_expanded", q, k, k_pe, v)
    a = _Expanded(q, k, k_pe, v, cu_q, cu_q_dev, cu_k, cu_k_dev, scale)
    with _OnDevice(q, stream) as s:
        shape = (a.Tq, a.Hq, a.D)
        if out is None:
            out = torch.empty(shape, dtype=q.dtype, device=a.device)
        else:
            _like(out, "out", shape, q.dtype, a.device)
        if lse is not None:
            _like(lse, "lse", shape[:2], torch.float32, a.device)
        elif want_lse:
            lse = torch.empty(shape[:2], dtype=torch.float32, device=a.device)
        if workspace is None:
            nb = int(lib().kpool_attend_expanded_workspace_bytes(*a.lens))
            workspace = torch.empty(nb, dtype=torch.uint8, device=a.device) if nb else None
        rc = lib().kpool_attend_expanded(*a.rows, *a.cu, _at(workspace), _bytes(workspace, a.device), _at(out), _at(lse), s)
    _check(rc, "kpool_attend_expanded")
    return out, lse


def attend_expanded_backward_workspace_bytes(cu_q, cu_k, Hq: int, Hkv: int, D: int, P: int) -> int:
    """Workspace of attend_expanded_backward for these sequences."""
    return _expanded_bytes("kpool_attend_expanded_backward_workspace_bytes", cu_q, cu_k, Hq, Hkv, D, P)


def attend_expanded_backward(d_o, q, k, k_pe, v, o, lse, cu_q, cu_q_dev, cu_k=None, cu_k_dev=None,
                             scale: float | None = None, workspace=None, dq=None, dk=None, dk_pe=None, dv=None, stream=None):
    """Gradients (dq, dk, dk_pe, dv) of attend_expanded: d_o is the gradient of o [Tq, Hq, D]; o and lse are
    what attend_expanded returned (want_lse=True); the rest are its arguments.  dq is [Tq, Hq, D + P], dk and
    dv [Tk, Hkv, D], dk_pe [Tk, P], in bf16."""
    import torch
    a = _Expanded(q, k, k_pe, v, cu_q, cu_q_dev, cu_k, cu_k_dev, scale)
    rows, keys = (a.Tq, a.Hq, a.D), (a.Tk, a.Hkv, a.D)
    _like(d_o, "d_o", rows, q.dtype, q.device)
    _like(o, "o", rows, q.dtype, q.device)
    _like(lse, "lse", rows[:2], torch.float32, q.device)
    with _OnDevice(q, stream) as s:
        out = []
        for t, name, shape in ((dq, "dq", (a.Tq, a.Hq, a.D + a.P)), (dk, "dk", keys), (dk_pe, "dk_pe", (a.Tk, a.P)),
                               (dv, "dv", keys)):
            if t is None:
                t = torch.empty(shape, dtype=q.dtype, device=q.device)
            else:
                _like(t, name, shape, q.dtype, q.device)
            out.append(t)
        if workspace is None:
            nb = int(lib().kpool_attend_expanded_backward_workspace_bytes(*a.lens))
            workspace = torch.empty(nb, dtype=torch.uint8, device=a.device) if nb else None
        rc = lib().kpool_attend_expanded_backward(_at(d_o), *a.rows, _at(o), _at(lse), *a.cu, _at(workspace),
                                                  _bytes(workspace, q.device), *(_at(t) for t in out), s)
    _check(rc, "kpool_attend_expanded_backward")
    return tuple(out)


class _Latent:
    """The arguments that both forms of the latent attention share, checked."""

    def __init__(self, q, cache, rank, cu_q, cu_q_dev, k_lens, scale, page_table, k_starts):
        import torch
        codes = (torch.bfloat16, torch.int16)
        self.device = device = q.device
        tq, self.H, width, qs = _heads(q, "q", device, codes)
        self.R, self.P = rank, width - rank
        if not 0 < rank <= width:
            raise ValueError(f"rank must be in 1 .. {width}, the values of a head of q")
        if cache.dtype not in codes or cache.device != device or cache.shape[-1:] != (width,):
            raise ValueError(f"cache must be a bfloat16 (or int16) tensor with rows of {width} values on {device}")
        if (page_table is None) == (k_starts is None):
            raise ValueError("give one of page_table and k_starts")
        self.cu_q = cu = np.ascontiguousarray(cu_q, dtype=np.int32)
        if cu.ndim != 1 or len(cu) < 2:
            raise ValueError("cu_q must be 1-dimensional with nseq + 1 entries")
        self.nseq, self.Tq = len(cu) - 1, int(cu[-1])
        _like(cu_q_dev, "cu_q_dev", cu.shape, torch.int32, device)
        _like(k_lens, "k_lens", (self.nseq,), torch.int32, device)
        if tq < self.Tq:
            raise ValueError("q has fewer tokens than its cumulative lengths say")
        rows, per_seq, page = cache.shape[0], 0, 1
        stride = cache.stride()
        if page_table is not None:
            if cache.dim() != 3 or page_table.dim() != 2:
                raise ValueError("with a page table the cache is [pages, page_size, R + P], the table [nseq, pages]")
            page, per_seq = cache.shape[1], page_table.shape[1]
            _like(page_table, "page_table", (self.nseq, per_seq), torch.int32, device)
            if rows > 1 and page > 0 and stride[0] != page * stride[1] and page > 1:
                raise ValueError("the pages of the cache must follow one another")
            row_stride = stride[1] if page > 1 else stride[0] if rows > 1 else width
            rows *= page
        else:
            if cache.dim() != 2:
                raise ValueError("with k_starts the cache is [rows, R + P]")
            _like(k_starts, "k_starts", (self.nseq,), torch.int32, device)
            row_stride = stride[0] if rows > 1 else width
        if stride[-1] != 1 and width > 1:
            raise ValueError("the values of a row of the cache must be contiguous")
        self.cu_ptr = _host_address(cu)
        # (a table of no pages has no address, but is one: nothing is read behind the address given for it)
        table = k_lens.data_ptr() if page_table is not None and per_seq == 0 else _at(page_table)
        self.keys = (q.data_ptr(), qs, cache.data_ptr() if rows else None, row_stride, rows, table, per_seq, page,
                     _at(k_starts), k_lens.data_ptr())
        self.cu = (self.cu_ptr, cu_q_dev.data_ptr(), self.nseq, self.H, self.R, self.P, scale)

    def outputs(self, q, out, lse, want_lse):
        import torch
        shape = (self.Tq, self.H, self.R)
        if out is None:
            out = torch.empty(shape, dtype=q.dtype, device=self.device)
        else:
            _like(out, "out", shape, q.dtype, self.device)
        if lse is not None:
            _like(lse, "lse", shape[:2], torch.float32, self.device)
        elif want_lse:
            lse = torch.empty(shape[:2], dtype=torch.float32, device=self.device)
        return out, lse


def _latent_bytes(fn, *args):
    nb = int(getattr(lib(), fn)(*args))
    msg = lib().kpool_last_error().decode()
    if msg:
        raise KpoolError(fn, KPOOL_EINVAL, msg)
    return nb


def attend_latent_workspace_bytes(cu_q, max_len: int, H: int, R: int, P: int) -> int:
    """Workspace of attend_latent for these sizes (0 where it needs none)."""
    _int32(max_len=max_len, H=H, R=R, P=P)
    cu_q, qp = _host_i32(cu_q)
    return _latent_bytes("kpool_attend_latent_workspace_bytes", qp, len(cu_q) - 1, max_len, H, R, P)


def attend_latent(q, cache, rank: int, cu_q, cu_q_dev, k_lens, max_len: int, scale: float, page_table=None,
                  k_starts=None, out=None, want_lse: bool = False, lse=None, workspace=None, stream=None):
    """Latent attention, absorbed: query rows over the cached tokens they see: (o, lse or None).

    q bf16 [Tq, H, R + P] (any token stride), R being rank; the cache holds one row of R + P values a
    token, which is every head's key and whose first R are the value: [pages, page_size, R + P] with
    page_table int32 [nseq, pages], the cache's pages one behind another (a slice of interleaved ones is
    refused), or [rows, R + P] with k_starts int32 [nseq], the sequences' first rows.  k_lens int32
    [nseq], on the device: each sequence's tokens, of which its queries (cu_q, host and device) are the
    last, at most max_len.  A captured call reads lengths, pages and starts anew at each replay.  o is
    bf16 [Tq, H, R].  Serving only: there is no backward pass, and tensors that require gradients are
    refused where autograd would record the call."""
    _refuse_graph("attend_latent", q, cache)
    _int32(max_len=max_len)
    a = _Latent(q, cache, rank, cu_q, cu_q_dev, k_lens, scale, page_table, k_starts)
    with _OnDevice(q, stream) as s:
        out, lse = a.outputs(q, out, lse, want_lse)
        if workspace is None:
            import torch
            nb = int(lib().kpool_attend_latent_workspace_bytes(a.cu_ptr, a.nseq, max_len, a.H, a.R, a.P))
            workspace = torch.empty(nb, dtype=torch.uint8, device=a.device) if nb else None
        rc = lib().kpool_attend_latent(*a.keys, max_len, *a.cu, _at(workspace), _bytes(workspace, a.device), _at(out),
                                       _at(lse), s)
    _check(rc, "kpool_attend_latent")
    return out, lse


def attend_latent_selected_workspace_bytes(Tq: int, width: int, H: int, R: int, P: int) -> int:
    """Workspace of attend_latent_selected for these sizes (0 where it needs none)."""
    _int32(Tq=Tq, width=width, H=H, R=R, P=P)
    return _latent_bytes("kpool_attend_latent_selected_workspace_bytes", Tq, width, H, R, P)


def attend_latent_selected(q, cache, rank: int, token_ids, cu_q, cu_q_dev, k_lens, scale: float, page_table=None,
                           k_starts=None, out=None, want_lse: bool = False, lse=None, workspace=None, stream=None):
    """attend_latent over the tokens each row selected: token_ids int32 [Tq, width], sequence-local
    ids as expand gives them; entries that are negative or past the row stand for nothing."""
    _refuse_graph("attend_latent_selected", q, cache)
    import torch
    a = _Latent(q, cache, rank, cu_q, cu_q_dev, k_lens, scale, page_table, k_starts)
    if token_ids.dim() != 2:
        raise ValueError("token_ids must be [Tq, width]")
    width = token_ids.shape[1]
    _like(token_ids, "token_ids", (a.Tq, width), torch.int32, a.device)
    with _OnDevice(q, stream) as s:
        out, lse = a.outputs(q, out, lse, want_lse)
        if workspace is None:
            nb = int(lib().kpool_attend_latent_selected_workspace_bytes(a.Tq, width, a.H, a.R, a.P))
            workspace = torch.empty(nb, dtype=torch.uint8, device=a.device) if nb else None
        rc = lib().kpool_attend_latent_selected(*a.keys, _at(token_ids), width, *a.cu, _at(workspace),
                                                _bytes(workspace, a.device), _at(out), _at(lse), s)
    _check(rc, "kpool_attend_latent_selected")
    return out, lse


def _norm_rows(x, name):
    """x as rows: (rows, N, row stride, dtype code)."""
    import torch
    shape, dtype = x.shape, x.dtype
    if len(shape) != 2 or not x.is_cuda:
        raise ValueError(f"{name} must be a device tensor of rows [rows, N]")
    if dtype == torch.float32:
        code = KPOOL_DTYPE_F32
    elif dtype == torch.bfloat16 or dtype == torch.int16:
        code = KPOOL_DTYPE_BF16
    else:
        raise ValueError(f"{name} must be bfloat16 (or int16 bit patterns) or float32")
    rows, N = shape
    s0, s1 = x.stride()
    if N < 1 or (N > 1 and s1 != 1) or (rows > 1 and s0 < N):
        raise ValueError(f"{name} must hold contiguous rows that do not overlap")
    return rows, N, s0 if rows > 1 else N, code


def layer_norm(x, weight=None, bias=None, eps: float = 1e-6, out=None, want_stats: bool = False,
               stream=None):
    """Layer norm of the rows of x [rows, N] (bf16 or fp32, any row stride), with fp32 weight
    and bias [N] (None: ones, zeros).  Returns (y, mean, rstd); mean and rstd, fp32 [rows],
    are what layer_norm_backward reads, and None unless want_stats.  Autograd does not record the
    call (tensors that require gradients are refused where it would)."""
    import torch
    _refuse_graph("layer_norm", x, weight, bias)
    rows, N, stride, code = _norm_rows(x, "x")
    device = x.device
    if weight is not None:
        _like(weight, "weight", (N,), torch.float32, device)
    if bias is not None:
        _like(bias, "bias", (N,), torch.float32, device)
    if out is not None:
        _like(out, "out", (rows, N), x.dtype, device)
    with _OnDevice(x, stream) as s:
        if out is None:
            out = torch.empty_strided((rows, N), (N, 1), dtype=x.dtype, device=device)
        mean = rstd = None
        if want_stats:
            mean, rstd = x.new_empty((2, rows), dtype=torch.float32).unbind()
        rc = lib().kpool_layer_norm(x.data_ptr(), stride, _at(weight), _at(bias), rows, N, eps, code,
                                    out.data_ptr(), _at(mean), _at(rstd), s)
    _check(rc, "kpool_layer_norm")
    return out, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, want_dx: bool = True, want_dweight: bool = True,
                        want_dbias: bool = True, workspace=None, stream=None):
    """Gradients of layer_norm: (dx, dweight, dbias), each None where it is not wanted.  dy is
    like y; x, weight as in the forward call; mean, rstd from it.  A workspace of
    layer_norm_backward_workspace_bytes(rows, N) bytes may be passed in."""
    import torch
    rows, N, stride, code = _norm_rows(x, "x")
    _like(dy, "dy", (rows, N), x.dtype, x.device)
    if weight is not None:
        _like(weight, "weight", (N,), torch.float32, x.device)
    _like(mean, "mean", (rows,), torch.float32, x.device)
    _like(rstd, "rstd", (rows,), torch.float32, x.device)
    if not (want_dx or want_dweight or want_dbias):
        raise ValueError("no output is wanted")
    with _OnDevice(x, stream) as s:
        dx = x.new_empty((rows, N)) if want_dx else None
        dw = x.new_empty(N, dtype=torch.float32) if want_dweight else None
        db = x.new_empty(N, dtype=torch.float32) if want_dbias else None
        if workspace is None and (want_dweight or want_dbias):
            workspace = torch.empty(layer_norm_backward_workspace_bytes(rows, N), dtype=torch.uint8,
                                    device=x.device)
        rc = lib().kpool_layer_norm_backward(_at(dy), _at(x), stride, _at(weight), _at(mean), _at(rstd), rows,
                                             N, code, _at(workspace), _bytes(workspace, x.device), _at(dx),
                                             _at(dw), _at(db), s)
    _check(rc, "kpool_layer_norm_backward")
    return dx, dw, db


def layer_norm_backward_workspace_bytes(rows: int, N: int) -> int:
    return int(lib().kpool_layer_norm_backward_workspace_bytes(rows, N))


def rotary_frequencies(pairs: int, base: float = 10000.0, scale: float = 1.0, trained: int | None = None,
                       fast: float = 32.0, slow: float = 1.0, device="cuda"):
    """Frequencies of rotary positions, fp64 [pairs] in radians a token, and the factor on the
    rotated values: (freqs, factor).

    Pair j of n turns by base^(-j / n) a token.  For contexts `scale` times as long as the
    `trained` length (YaRN, Peng et al. 2023, section 3): pairs that make more than `fast` turns
    within the trained length keep their frequency, those that make less than `slow` turns are
    slowed by `scale`, and those between are mixed linearly; factor is 0.1 ln(scale) + 1.  With
    trained=None every pair is slowed alike (linear interpolation), and factor is 1."""
    import torch
    if pairs < 1 or not base > 0 or not scale >= 1 or not fast > slow or (trained is not None and trained < 1):
        raise ValueError("need pairs >= 1, base > 0, scale >= 1, fast > slow and trained >= 1")
    freqs = base ** (-np.arange(pairs, dtype=np.float64) / pairs)
    factor = 1.0
    if scale > 1 and trained is None:
        freqs = freqs / scale
    elif scale > 1:
        turns = trained * freqs / (2 * np.pi)
        keep = np.clip((turns - slow) / (fast - slow), 0.0, 1.0)
        freqs = freqs * (keep + (1.0 - keep) / scale)
        factor = 0.1 * float(np.log(scale)) + 1.0
    return torch.from_numpy(freqs).to(device), factor


def _rotary(fn, x, positions, freqs, begin, interleaved, factor, out, stream, inverse):
    import torch
    _int32(begin=begin)
    dtype, device = x.dtype, x.device
    shape = x.shape
    if len(shape) == 2:
        rows, D = shape
        heads, (s0, s2) = 1, x.stride()
        s1 = D
    elif len(shape) == 3:
        rows, heads, D = shape
        s0, s1, s2 = x.stride()
    else:
        raise ValueError("x must be [rows, heads, D] or [rows, D]")
    if not x.is_cuda or heads < 1 or (s2 != 1 and D > 1) or (s1 != D and heads > 1):
        raise ValueError("x must be a device tensor with the heads of a row contiguous")
    if dtype == torch.float32:
        code = KPOOL_DTYPE_F32
    elif dtype == torch.bfloat16 or dtype == torch.int16:
        code = KPOOL_DTYPE_BF16
    else:
        raise ValueError("x must be bfloat16 (or int16 bit patterns) or float32")
    if rows > 1 and s0 < heads * D:
        raise ValueError("x must hold rows that do not overlap")
    _like(positions, "positions", (rows,), torch.int32, device)
    if freqs.dim() != 1:
        raise ValueError("freqs must be [pairs]")
    pairs = freqs.shape[0]
    _like(freqs, "freqs", (pairs,), torch.float64, device)
    y0 = heads * D
    if out is not None:
        if out.shape != shape or out.dtype != dtype or out.device != device or (D > 1 and out.stride(-1) != 1) or (
                heads > 1 and out.stride(1) != D):
            raise ValueError(f"out must be like x: {dtype} {tuple(shape)} on {device}, the heads of a row contiguous")
        if rows > 1:
            y0 = out.stride(0)
    flags = (KPOOL_ROTARY_INTERLEAVED if interleaved else 0) | (KPOOL_ROTARY_INVERSE if inverse else 0)
    with _OnDevice(x, stream) as s:
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=device)
        rc = lib().kpool_rotary(x.data_ptr(), s0 if rows > 1 else heads * D, positions.data_ptr(), freqs.data_ptr(),
                                rows, heads, D, begin, pairs, factor, code, flags, out.data_ptr(), y0, s)
    _check(rc, "kpool_rotary")
    return out


def rotary(x, positions, freqs, begin: int = 0, interleaved: bool = False, factor: float = 1.0, out=None, stream=None):
    """Rotary positions: pairs of each head's values of x [rows, heads, D] or [rows, D] (bf16 or fp32, any
    row stride) turned by positions[r] * freqs[j], times factor; the head's other values copied.

    positions int32 [rows], freqs fp64 [pairs] (rotary_frequencies makes them).  Pair j is the values
    begin + j and begin + pairs + j of a head, or, interleaved, begin + 2 j and begin + 2 j + 1.
    out may be x itself (in place) or a slice of wider rows.  Autograd does not record the call (tensors
    that require gradients are refused where it would); rotary_backward has its gradient."""
    _refuse_graph("rotary", x)
    return _rotary("rotary", x, positions, freqs, begin, interleaved, factor, out, stream, False)


def rotary_backward(dy, positions, freqs, begin: int = 0, interleaved: bool = False, factor: float = 1.0, out=None,
                    stream=None):
    """Gradient of rotary: dx, the values of dy turned back.  The other arguments are the forward call's."""
    return _rotary("rotary_backward", dy, positions, freqs, begin, interleaved, factor, out, stream, True)


def _bytes(workspace, device):
    """Size of a caller's workspace (0 for none)."""
    if workspace is None:
        return 0
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace.numel() * workspace.element_size()


def profile_enable(on: bool = True):
    _check(lib().kpool_profile_enable(1 if on else 0), "kpool_profile_enable")


def profile_collect():
    """{kind: (ms, launches)} accumulated since the last collect."""
    out = {}
    for kinds, fn in ((PROFILE_KINDS, "kpool_profile_collect"),
                      (LAYER_PROFILE_KINDS, "kpool_layer_profile_collect")):
        ms = (ctypes.c_double * len(kinds))()
        n = (ctypes.c_int64 * len(kinds))()
        _check(getattr(lib(), fn)(ms, n), fn)
        out.update((k, (ms[i], int(n[i]))) for i, k in enumerate(kinds))
    return out


def row_range(cu, q_lo: int, q_hi: int):
    """(cu_q, cu_k) of the attention calls for the rows [q_lo, q_hi) of a packed batch: each
    sequence's rows in the range, and its keys up to the last of them."""
    cu = np.asarray(cu, dtype=np.int32)
    if not 0 <= q_lo <= q_hi <= int(cu[-1]):
        raise ValueError("need 0 <= q_lo <= q_hi <= T")
    return np.clip(cu, q_lo, q_hi) - np.int32(q_lo), np.minimum(cu, np.int32(q_hi))


# ---------------------------------------------------------------------------
# Whole path on one batch
# ---------------------------------------------------------------------------

class Selector:
    """Pool -> score/top-k -> expand for one packed batch layout (device tensors in, out).

    Holds the device copies of cu_seqlens / cu_pools and a workspace sized
    for the row range; `run` enqueues the three library calls on one stream.
    By default the workspace is one chunk buffer, so all fp32 scores in flight stay
    within the 2 GiB cap; overlap=True sizes it for two chunk buffers and runs the
    chunk loop with KPOOL_FLAG_OVERLAP (two chunks in flight on two streams);
    workspace_cap caps the workspace (smaller chunks); tail=True runs every step in
    tail mode (KPOOL_FLAG_TAIL).  rotary=(freqs, begin, interleaved, factor) gives `run`'s queries and
    keys rotary positions, counted from each sequence's start, before they meet.  `attend` is the
    attention of the same rows over what the last run selected.
    """

    def __init__(self, cu_seqlens, kpool: int, budget: int, H: int, D: int, device="cuda",
                 q_lo: int = 0, q_hi: int | None = None, workspace_cap: int | None = None,
                 scale: float | None = None, overlap: bool = False, tail: bool = False, rotary=None):
        import torch
        self.cu = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int32))
        self.T = int(self.cu[-1])
        self.kpool, self.budget, self.H, self.D = kpool, budget, H, D
        self.q_lo = q_lo
        self.q_hi = self.T if q_hi is None else q_hi
        self.overlap = overlap
        self.tail = tail
        self.cu_pools, self.max_pools, self.P_tot = count_pools(self.cu, kpool, tail)
        self.cu_dev = torch.from_numpy(self.cu).to(device)
        self.cu_pools_dev = torch.from_numpy(self.cu_pools).to(device)
        self.scale = float(np.float32(1.0) / np.sqrt(np.float32(D))) if scale is None else scale
        nb = workspace_bytes(self.q_lo, self.q_hi, self.max_pools, 2 if overlap else 1)
        if workspace_cap is not None:
            nb = min(nb, workspace_cap)
        self.workspace = torch.empty(max(nb, 16), dtype=torch.uint8, device=device)
        rows = self.q_hi - self.q_lo
        self.kp = torch.empty((self.P_tot, D), dtype=torch.int16, device=device)
        self.pool_ids = torch.empty((rows, budget), dtype=torch.int32, device=device)
        self.token_ids = torch.empty((rows, budget * kpool + (kpool - 1 if tail else 0)),
                                     dtype=torch.int32, device=device)
        self.k_normed = None
        # the rows' sequences for the attention: their queries and the keys up to the last row
        self.attend_cu = row_range(self.cu, self.q_lo, self.q_hi)
        self.attend_cu_dev = tuple(torch.from_numpy(c).to(device) for c in self.attend_cu)
        self.rotary = rotary
        if rotary is not None:
            local = np.arange(self.T, dtype=np.int32) - np.repeat(self.cu[:-1], np.diff(self.cu))
            self.positions = torch.from_numpy(local.astype(np.int32)).to(device)
            self.q_turned = torch.empty((rows, H, D), dtype=torch.int16, device=device)  # (the range's rows)
            self.k_turned = torch.empty((self.T, D), dtype=torch.int16, device=device)

    @property
    def workspace_bytes(self) -> int:
        return self.workspace.numel()

    def chunk_rows(self, overlap: bool | None = None) -> int:
        """Rows per chunk of the chunk loop with this workspace (the library's plan)."""
        overlap = self.overlap if overlap is None else overlap
        return chunk_rows(self.max_pools, self.workspace_bytes, overlap, self.tail)[0]

    def chunk_buffers(self, overlap: bool | None = None) -> int:
        overlap = self.overlap if overlap is None else overlap
        return chunk_rows(self.max_pools, self.workspace_bytes, overlap, self.tail)[1]

    def run(self, q, k, w, scores_out=None, stream=None, overlap: bool | None = None, g=None,
            ape=None, k_norm=None):
        """One pass of the path; with gate scores g and slot embeddings ape the keys are
        pooled by the gated compression, otherwise by the mean.  With k_norm = (weight, bias,
        eps), k is the key projection's output and passes that layer norm first (its rows may
        then be a slice of a wider projection).  A selector with rotary positions turns q and the
        (normalised) keys next, into buffers of its own; gate scores are left as they are."""
        import torch
        overlap = self.overlap if overlap is None else overlap
        if k_norm is not None:
            weight, bias, eps = k_norm
            if k.dim() != 2 or k.shape[0] < self.T or k.element_size() != 2:
                raise ValueError(f"k must be bfloat16 (or int16 bit patterns) with {self.T} rows")
            if self.k_normed is None:  # (for good: a captured run keeps writing there)
                with _on(stream):
                    self.k_normed = k.new_empty((self.T, self.D))
            g = None if g is None else g[:self.T]
            with torch.no_grad():  # (ids have no gradients)
                k = layer_norm(k[:self.T], weight, bias, eps, out=self.k_normed.view(k.dtype), stream=stream)[0]
        first = 0
        if self.rotary is not None:
            q, k = self._turn(q, k, stream)
            first = self.q_lo
            g = None if g is None else g[:self.T]
        if g is not None:
            pool_keys_gated(k, g, ape, self.cu, self.cu_dev, self.cu_pools_dev, self.kpool,
                            out=self.kp, stream=stream, tail=self.tail)
        else:
            pool_keys(k, self.cu, self.cu_dev, self.cu_pools_dev, self.kpool, out=self.kp,
                      stream=stream, tail=self.tail)
        _score_topk(q, first, self.kp, w, self.cu, self.cu_dev, self.kpool, self.budget, self.q_lo, self.q_hi,
                    scale=self.scale, workspace=self.workspace, pool_ids=self.pool_ids, scores_out=scores_out,
                    want_scores=False, overlap=overlap, stream=stream, tail=self.tail)
        expand(self.pool_ids, self.cu, self.cu_dev, self.kpool, self.budget, self.q_lo, self.q_hi,
               out=self.token_ids, stream=stream, tail=self.tail)
        return {"kp": self.kp, "pool_ids": self.pool_ids, "token_ids": self.token_ids}

    def _turn(self, q, k, stream):
        """Index queries (the rows' own) and keys at their positions, in the selector's buffers."""
        import torch
        if q.shape != (self.T, self.H, self.D) or q.element_size() != 2 or k.dim() != 2 or k.shape[0] < self.T:
            raise ValueError(f"need q [{self.T}, {self.H}, {self.D}] and k with {self.T} rows in bfloat16 (or int16)")
        freqs, begin, interleaved, factor = self.rotary
        how = dict(begin=begin, interleaved=interleaved, factor=factor, stream=stream)
        rows = slice(self.q_lo, self.q_hi)
        with torch.no_grad():  # (ids have no gradients)
            rotary(q[rows], self.positions[rows], freqs, out=self.q_turned.view(q.dtype), **how)
            rotary(k[:self.T], self.positions, freqs, out=self.k_turned.view(k.dtype), **how)
        return self.q_turned, self.k_turned

    def attend(self, q, k, v, scale: float | None = None, out=None, want_lse: bool = False, stream=None):
        """Attention of the selector's rows over the tokens the last run selected for them:
        (o, lse or None), one row per row of [q_lo, q_hi).

        q bf16 [T, Hq, D], k and v bf16 [T, Hkv, D] (the attention's own, of any token stride),
        of which rows [q_lo, q_hi) and, for keys, the rows before them are used.  Where every
        sequence has at most `budget` pools, every row selected all it sees, and the attention
        over whole keys gives the same without reading lists (2048 tokens, 32 heads over 2:
        202 us by lists, 60 us whole)."""
        (cu_q, cu_k), (cqd, ckd) = self.attend_cu, self.attend_cu_dev
        args = (cu_q, cqd, cu_k, ckd)
        q, keys = q[self.q_lo:self.q_hi], int(cu_k[-1])
        kw = dict(scale=scale, out=out, want_lse=want_lse, stream=stream)
        if self.max_pools <= self.budget:
            return attend(q, k[:keys], v[:keys], *args, **kw)
        return attend_selected(q, k[:keys], v[:keys], self.token_ids, *args, **kw)
