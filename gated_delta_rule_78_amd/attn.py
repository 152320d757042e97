"""The softmax-attention layers between KDA layers (``include/kda_attn.h``).

    head_rope_fwd(q, k, inv_freq, positions) -> (q_out, k_out)   norm of every head and rotation
    head_rope_bwd(q, k, inv_freq, dq_out, dk_out, positions)     gradients of rows and weights
        -> (dq, dk, dq_weight, dk_weight)
    kv_append(q, k, v, k_cache, v_cache, block_table, kv_lens, inv_freq) -> q_out
                                                                 new tokens into a paged cache
    paged_attn(q, k_cache, v_cache, block_table, kv_lens) -> o   attention of new tokens over it
"""
import ctypes
import functools

import torch

from . import _DTYPES, _check, _check_workspace, _nbytes, _workspace, library
from ._launch import check, on_gpu, ptr, raw_stream, scope

ROPE_MAX_D = 1024    # KDA_ROPE_MAX_D of include/kda_attn.h


class RowStrides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("h", ctypes.c_int64), ("t", ctypes.c_int64)]


class PageStrides(ctypes.Structure):
    _fields_ = [("p", ctypes.c_int64), ("h", ctypes.c_int64), ("t", ctypes.c_int64)]


class HeadRopeDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("Hq", ctypes.c_int64), ("Hk", ctypes.c_int64), ("T", ctypes.c_int64),
                ("d", ctypes.c_int64), ("rot", ctypes.c_int64), ("q", RowStrides), ("k", RowStrides),
                ("q_out", RowStrides), ("k_out", RowStrides), ("dq", RowStrides), ("dk", RowStrides),
                ("dtype", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("norm", ctypes.c_int32),
                ("eps", ctypes.c_float), ("rope_scale", ctypes.c_float)]


class KvAppendDesc(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("Hq", ctypes.c_int64), ("Hk", ctypes.c_int64), ("T", ctypes.c_int64),
                ("dk", ctypes.c_int64), ("dv", ctypes.c_int64), ("rot", ctypes.c_int64), ("pages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("max_pages", ctypes.c_int64), ("table_stride", ctypes.c_int64),
                ("q", RowStrides), ("k", RowStrides), ("v", RowStrides), ("q_out", RowStrides), ("k_cache", PageStrides),
                ("v_cache", PageStrides), ("in_dtype", ctypes.c_int32), ("packed", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("norm", ctypes.c_int32), ("eps", ctypes.c_float),
                ("rope_scale", ctypes.c_float)]


class PagedAttnDesc(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("Hq", ctypes.c_int64), ("Hk", ctypes.c_int64), ("T", ctypes.c_int64),
                ("dk", ctypes.c_int64), ("dv", ctypes.c_int64), ("pages", ctypes.c_int64), ("page_size", ctypes.c_int64),
                ("max_pages", ctypes.c_int64), ("table_stride", ctypes.c_int64), ("window", ctypes.c_int64),
                ("q", RowStrides), ("o", RowStrides), ("k_cache", PageStrides), ("v_cache", PageStrides),
                ("packed", ctypes.c_int32), ("scale", ctypes.c_float)]


_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = library()
        P, Z, I = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
        H, K = ctypes.POINTER(HeadRopeDesc), ctypes.POINTER(KvAppendDesc)
        lib.kda_head_rope_fwd.argtypes = [H] + [P] * 9
        lib.kda_head_rope_fwd.restype = I
        lib.kda_head_rope_bwd_workspace_bytes.argtypes = [H]
        lib.kda_head_rope_bwd_workspace_bytes.restype = Z
        lib.kda_head_rope_bwd.argtypes = [H] + [P] * 13 + [Z, P]
        lib.kda_head_rope_bwd.restype = I
        lib.kda_kv_append.argtypes = [K] + [P] * 13
        lib.kda_kv_append.restype = I
        A = ctypes.POINTER(PagedAttnDesc)
        lib.kda_paged_attn_workspace_bytes.argtypes = [A]
        lib.kda_paged_attn_workspace_bytes.restype = Z
        lib.kda_paged_attn.argtypes = [A] + [P] * 9 + [Z, P]
        lib.kda_paged_attn.restype = I
        _lib = lib
    return _lib


def _check_rows(name, t, index, dtype, shape):
    """``t`` must be a ``dtype`` tensor of ``shape`` on GPU ``index``, its last dimension contiguous."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or (t.stride(-1) != 1 and t.shape[-1] > 1):
        raise ValueError("%s must be a %s tensor of shape %s on %s, its last dimension contiguous (got %s %s %s, strides %s)"
                         % (name, dtype, tuple(shape), "cuda:%d" % index if index >= 0 else "the inputs' device", t.dtype,
                            tuple(t.shape), t.device, t.stride()))


def _outer(t):
    """Strides (b, h, t) of [B,H,T,d] or packed [H,T,d] rows."""
    if t is None:
        return (0, 0, 0)
    s = t.stride()
    return s[:3] if len(s) == 4 else (0, s[0], s[1])


@functools.lru_cache(maxsize=1024)
def _rope_desc(B, Hq, Hk, T, d, rot, strides, dtype, interleaved, norm, eps, rope_scale):
    """The call's descriptor: nothing but its arguments, so calls of one shape share it."""
    return HeadRopeDesc(B, Hq, Hk, T, d, rot, *(RowStrides(*s) for s in strides), _DTYPES[dtype], interleaved, norm, eps,
                        rope_scale)


def _rope_inputs(fn, q, k, inv_freq, positions, q_weight, k_weight, norm):
    """Checks the inputs that both directions share; returns (a row tensor, its GPU, B, Hq, Hk, T, d, rot)."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("one of q and k is required")
    if x.dtype not in _DTYPES:
        raise ValueError("unsupported dtype %s" % x.dtype)
    if x.dim() not in (3, 4):
        raise ValueError("rows must be [B,H,T,d] or [H,T,d] (got shape %s)" % (tuple(x.shape),))
    index, shape = x.get_device(), x.shape
    *b, _, T, d = shape
    Hq, Hk = (0 if t is None or t.dim() < 3 else t.shape[-3] for t in (q, k))
    for name, t, H in (("q", q, Hq), ("k", k, Hk)):
        if t is not None:
            _check_rows(name, t, index, x.dtype, (*b, H, T, d))
    rot = 0
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        check("inv_freq", inv_freq, index, torch.float32, (rot // 2,))
    if positions is not None:
        check("positions", positions, index, torch.int32, (*b, T))
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            if not norm:
                raise ValueError("%s goes with norm" % name)
            check(name, w, index, torch.float32, (d,))
    on_gpu(fn, x)
    return x, index, b[0] if b else 1, Hq, Hk, T, d, rot


def head_rope_fwd(q, k, inv_freq, positions=None, *, interleaved=False, rope_scale=1.0, q_weight=None, k_weight=None,
                  norm=True, eps=1e-6, q_out=None, k_out=None, stream=None):
    """Norm of every head of q and k and their rotation by position, through ``kda_head_rope_fwd``.

    q, k: [B,Hq,T,d], [B,Hk,T,d] or packed [H,T,d], bf16 or fp32, any strides with contiguous
    channels (slices of a projection's output are read where they are); either may be None.
    inv_freq: fp32 frequencies of the rotated pairs, [rot / 2], or None (no rotation); positions:
    int32 [B,T] (packed [T]), or None (0 .. T-1). The first rot channels turn in pairs
    (i, i + rot/2), or (2i, 2i + 1) with ``interleaved``, by positions * inv_freq, times rope_scale.
        y = weight * x / sqrt(mean(x^2) + eps)      (norm False: x itself; weights [d] fp32 or None)
    Returns (q_out, k_out) in the inputs' type, their dimensions in memory in the inputs' order;
    None for an input that was not given. Caller-supplied outputs are checked like the inputs."""
    x, index, B, Hq, Hk, T, d, rot = _rope_inputs("head_rope_fwd", q, k, inv_freq, positions, q_weight, k_weight, norm)
    for name, o, t in (("q_out", q_out, q), ("k_out", k_out, k)):
        if o is not None:
            if t is None:
                raise ValueError("%s goes with %s" % (name, name[0]))
            _check_rows(name, o, index, t.dtype, t.shape)
    with scope(index, stream):
        if q_out is None and q is not None:
            q_out = torch.empty_like(q)
        if k_out is None and k is not None:
            k_out = torch.empty_like(k)
        desc = _rope_desc(B, Hq, Hk, T, d, rot, (_outer(q), _outer(k), _outer(q_out), _outer(k_out), (0, 0, 0), (0, 0, 0)),
                          x.dtype, bool(interleaved), bool(norm), float(eps), float(rope_scale))
        st = (_lib or _library()).kda_head_rope_fwd(desc, ptr(q), ptr(k), ptr(q_weight), ptr(k_weight), ptr(inv_freq),
                                                    ptr(positions), ptr(q_out), ptr(k_out), raw_stream(index, stream))
    _check("kda_head_rope_fwd", st)
    return q_out, k_out


def head_rope_bwd(q, k, inv_freq, dq_out, dk_out, positions=None, *, interleaved=False, rope_scale=1.0, q_weight=None,
                  k_weight=None, norm=True, eps=1e-6, workspace=None, stream=None):
    """Backward of ``head_rope_fwd`` through ``kda_head_rope_bwd``.

    Inputs as the forward's; dq_out, dk_out: gradients of its outputs, in their shape and type, any
    strides. Returns (dq, dk, dq_weight, dk_weight): rows in their input's type, weight gradients [d]
    fp32; None for each input that was not given."""
    x, index, B, Hq, Hk, T, d, rot = _rope_inputs("head_rope_bwd", q, k, inv_freq, positions, q_weight, k_weight, norm)
    for name, g, t in (("dq_out", dq_out, q), ("dk_out", dk_out, k)):
        if (g is None) != (t is None):
            raise ValueError("%s goes with %s" % (name, name[1]))
        if g is not None:
            _check_rows(name, g, index, t.dtype, t.shape)
    if workspace is not None:
        _check_workspace(workspace, x.device)
    sums = q_weight is not None or k_weight is not None
    lib = _lib or _library()
    with scope(index, stream):
        dq = torch.empty_like(q) if q is not None else None
        dk = torch.empty_like(k) if k is not None else None
        dwq = torch.empty_like(q_weight) if q_weight is not None and q is not None else None
        dwk = torch.empty_like(k_weight) if k_weight is not None and k is not None else None
        desc = _rope_desc(B, Hq, Hk, T, d, rot, (_outer(q), _outer(k), _outer(dq_out), _outer(dk_out), _outer(dq), _outer(dk)),
                          x.dtype, bool(interleaved), bool(norm), float(eps), float(rope_scale))
        workspace = _workspace(lib.kda_head_rope_bwd_workspace_bytes(desc) if sums else 0, workspace, x.device)
        st = lib.kda_head_rope_bwd(desc, ptr(q), ptr(k), ptr(q_weight), ptr(k_weight), ptr(inv_freq), ptr(positions),
                                   ptr(dq_out), ptr(dk_out), ptr(dq), ptr(dk), ptr(dwq), ptr(dwk), ptr(workspace),
                                   _nbytes(workspace), raw_stream(index, stream))
    _check("kda_head_rope_bwd", st)
    return dq, dk, dwq, dwk


def _cache_inputs(index, first, cu_seqlens, kv_lens, block_table):
    """Checks what tells sequences and pages apart; returns (N, packed)."""
    packed = cu_seqlens is not None
    if first.dim() != (3 if packed else 4):
        raise ValueError("rows must be [H,T,d] with cu_seqlens, [N,H,T,d] without (got shape %s)" % (tuple(first.shape),))
    N = cu_seqlens.numel() - 1 if packed else first.shape[0]
    if packed:
        check("cu_seqlens", cu_seqlens, index, torch.int32, (N + 1,))
    check("kv_lens", kv_lens, index, torch.int32, (N,))
    _check_rows("block_table", block_table, index, torch.int32, (N, block_table.shape[-1]))
    return N, packed


@functools.lru_cache(maxsize=1024)
def _append_desc(N, Hq, Hk, T, dk, dv, rot, pages, page_size, max_pages, table_stride, rows, caches, dtype, packed,
                 interleaved, norm, eps, rope_scale):
    return KvAppendDesc(N, Hq, Hk, T, dk, dv, rot, pages, page_size, max_pages, table_stride,
                        *(RowStrides(*s) for s in rows), *(PageStrides(*s) for s in caches), _DTYPES[dtype], packed,
                        interleaved, norm, eps, rope_scale)


def kv_append(q, k, v, k_cache, v_cache, block_table, kv_lens, inv_freq=None, *, cu_seqlens=None, interleaved=False,
              rope_scale=1.0, q_weight=None, k_weight=None, norm=True, eps=1e-6, q_out=None, stream=None):
    """New tokens' keys and values into a paged cache, through ``kda_kv_append``: k normed and rotated
    at its position on the way, v copied; q (or None) normed and rotated into the returned q_out (bf16).

    q, k, v: [N,Hq,T,dk], [N,Hk,T,dk], [N,Hk,T,dv], T new tokens of each of N sequences, or packed
    [H,T,d] with cu_seqlens (int32 [N+1]); bf16 or fp32, any strides with contiguous channels.
    k_cache, v_cache: [pages,Hk,page_size,dk], [pages,Hk,page_size,dv] bf16, written in place, any
    strides with contiguous channels. block_table: int32 [N,max_pages]; position j of sequence s is
    row j % page_size of page block_table[s, j // page_size]. kv_lens: int32 [N], positions in use
    with the new tokens, which are each sequence's last. Norm and rotation as ``head_rope_fwd``."""
    if k.dtype not in _DTYPES:
        raise ValueError("unsupported dtype %s" % k.dtype)
    index, dt = k.get_device(), k.dtype
    N, packed = _cache_inputs(index, k, cu_seqlens, kv_lens, block_table)
    *b, Hk, T, dk = k.shape
    dv = v.shape[-1]
    _check_rows("k", k, index, dt, k.shape)
    _check_rows("v", v, index, dt, (*b, Hk, T, dv))
    Hq = 0
    if q is not None:
        Hq = q.shape[-3] if q.dim() >= 3 else 0
        _check_rows("q", q, index, dt, (*b, Hq, T, dk))
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages,Hk,page_size,dk] (got shape %s)" % (tuple(k_cache.shape),))
    pages, page_size = k_cache.shape[0], k_cache.shape[2]
    _check_rows("k_cache", k_cache, index, torch.bfloat16, (pages, Hk, page_size, dk))
    _check_rows("v_cache", v_cache, index, torch.bfloat16, (pages, Hk, page_size, dv))
    rot = 0
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        check("inv_freq", inv_freq, index, torch.float32, (rot // 2,))
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            if not norm:
                raise ValueError("%s goes with norm" % name)
            check(name, w, index, torch.float32, (dk,))
    if q_out is not None:
        if q is None:
            raise ValueError("q_out goes with q")
        _check_rows("q_out", q_out, index, torch.bfloat16, q.shape)
    on_gpu("kv_append", k)
    with scope(index, stream):
        if q_out is None and q is not None:
            q_out = torch.empty_like(q, dtype=torch.bfloat16)
        desc = _append_desc(N, Hq, Hk, T, dk, dv, rot, pages, page_size, block_table.shape[1], block_table.stride(0),
                            (_outer(q), _outer(k), _outer(v), _outer(q_out)),
                            (k_cache.stride()[:3], v_cache.stride()[:3]), dt, packed, bool(interleaved), bool(norm),
                            float(eps), float(rope_scale))
        st = (_lib or _library()).kda_kv_append(desc, ptr(q), ptr(k), ptr(v), ptr(q_weight), ptr(k_weight), ptr(inv_freq),
                                                ptr(cu_seqlens), ptr(kv_lens), ptr(block_table), ptr(q_out), ptr(k_cache),
                                                ptr(v_cache), raw_stream(index, stream))
    _check("kda_kv_append", st)
    return q_out


@functools.lru_cache(maxsize=1024)
def _attn_desc(N, Hq, Hk, T, dk, dv, pages, page_size, max_pages, table_stride, window, rows, caches, packed, scale):
    """The call's descriptor and the workspace it needs."""
    desc = PagedAttnDesc(N, Hq, Hk, T, dk, dv, pages, page_size, max_pages, table_stride, window,
                         *(RowStrides(*s) for s in rows), *(PageStrides(*s) for s in caches), packed, scale)
    return desc, _library().kda_paged_attn_workspace_bytes(desc)


def paged_attn(q, k_cache, v_cache, block_table, kv_lens, *, cu_seqlens=None, scale=None, window=0, o=None, lse=None,
               return_lse=False, workspace=None, stream=None):
    """Attention of new tokens over their sequences' positions in a paged cache, through ``kda_paged_attn``.

    q: [N,Hq,T,dk], T new tokens of each of N sequences, or packed [Hq,T,dk] with cu_seqlens (int32
    [N+1]); bf16, any strides in multiples of 8 with contiguous channels. k_cache [pages,Hk,page_size,dk],
    v_cache [pages,Hk,page_size,dv], block_table [N,max_pages], kv_lens [N] as ``kv_append`` left them:
    the new tokens are each sequence's last, token i of n at position kv_lens - n + i. It sees the positions
    up to its own, with ``window`` > 0 the last ``window`` of them.
        o = softmax(scale * q k^T) v,   lse = log sum exp(scale * q k^T)     (scale: default 1 / sqrt(dk))
    Query head h reads key head h // (Hq / Hk). Returns o [N,Hq,T,dv] (packed [Hq,T,dv]) bf16, its
    dimensions in memory in q's order; with ``return_lse`` (o, lse), lse fp32 [N,Hq,T] (packed [Hq,T]).
    A token that sees nothing has o = 0 and lse = -inf."""
    BF16 = torch.bfloat16
    index = q.get_device()
    N, packed = _cache_inputs(index, q, cu_seqlens, kv_lens, block_table)
    *b, Hq, T, dk = q.shape
    _check_rows("q", q, index, BF16, q.shape)
    if k_cache.dim() != 4 or v_cache.dim() != 4:
        raise ValueError("k_cache and v_cache must be [pages,Hk,page_size,d] (got shapes %s, %s)"
                         % (tuple(k_cache.shape), tuple(v_cache.shape)))
    pages, Hk, page_size, dv = v_cache.shape
    _check_rows("k_cache", k_cache, index, BF16, (pages, Hk, page_size, dk))
    _check_rows("v_cache", v_cache, index, BF16, v_cache.shape)
    if o is not None:
        _check_rows("o", o, index, BF16, (*b, Hq, T, dv))
    if lse is not None:
        check("lse", lse, index, torch.float32, (*b, Hq, T))
    if workspace is not None:
        _check_workspace(workspace, q.device)
    on_gpu("paged_attn", q)
    with scope(index, stream):
        if o is None:
            if dv == dk:
                o = torch.empty_like(q)
            else:      # q's order of dimensions: token-major rows stay so
                s = q.stride()
                o = (torch.empty(*b, T, Hq, dv, dtype=BF16, device=q.device).transpose(-3, -2) if s[-3] < s[-2]
                     else torch.empty(*b, Hq, T, dv, dtype=BF16, device=q.device))
        if lse is None and return_lse:
            lse = torch.empty(*b, Hq, T, dtype=torch.float32, device=q.device)
        desc, need = _attn_desc(N, Hq, Hk, T, dk, dv, pages, page_size, block_table.shape[1], block_table.stride(0),
                                int(window), (_outer(q), _outer(o)), (k_cache.stride()[:3], v_cache.stride()[:3]), packed,
                                float(dk ** -0.5 if scale is None else scale))
        workspace = _workspace(need, workspace, q.device)
        st = (_lib or _library()).kda_paged_attn(desc, ptr(q), ptr(k_cache), ptr(v_cache), ptr(cu_seqlens), ptr(kv_lens),
                                                 ptr(block_table), ptr(o), ptr(lse), ptr(workspace), _nbytes(workspace),
                                                 raw_stream(index, stream))
    _check("kda_paged_attn", st)
    return (o, lse) if return_lse else o
