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


def _strides(stride):
    return RowStrides(*(stride[:3] if len(stride) == 4 else (0, *stride[:2]) if stride else (0, 0, 0)))


# The entry points look their arguments over in one condition each, since a decode step's kernels take a
# few microseconds; only where it fails does _explain go through them one by one and raise.

def _explain(checks):
    for f, *args in checks:
        f(*args)
    raise ValueError("arguments do not go together")


@functools.lru_cache(maxsize=1024)
def _rope_desc(q, k, q_strides, k_strides, qo, ko, dq, dk, rot, dtype, interleaved, norm, eps, rope_scale):
    """The call's descriptor: nothing but its arguments, so calls of one shape share it."""
    x = q if q is not None else k
    B, T, d = (x[0] if len(x) == 4 else 1), x[-2], x[-1]
    return HeadRopeDesc(B, q[-3] if q is not None else 0, k[-3] if k is not None else 0, T, d, rot,
                        *(_strides(s) for s in (q_strides, k_strides, qo, ko, dq, dk)), _DTYPES[dtype], interleaved, norm,
                        eps, rope_scale)


@functools.lru_cache(maxsize=1024)
def _rope_bwd_desc(*shape):
    """The backward's descriptor and the workspace that weight gradients need."""
    desc = _rope_desc(*shape)
    return desc, _library().kda_head_rope_bwd_workspace_bytes(desc)


def _rope_inputs(fn, q, k, inv_freq, positions, q_weight, k_weight, norm):
    """Checks the inputs that both directions share; returns (shapes and strides of q and k, GPU, rot)."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("one of q and k is required")
    index, dt, shape = x.get_device(), x.dtype, x.shape
    rows, d = shape[:-3] + shape[-2:-1], shape[-1:]
    qs = ks = None
    qst = kst = ()
    ok = dt in _DTYPES and 3 <= len(shape) <= 4
    if q is not None:
        qs, qst = q.shape, q.stride()
        ok = ok and qst[-1] == 1
    if k is not None:
        ks, kst = k.shape, k.stride()
        ok = (ok and kst[-1] == 1 and k.dtype is dt and len(ks) == len(shape) and ks[:-3] == shape[:-3] and ks[-2:] == shape[-2:]
              and k.get_device() == index)
    if positions is not None:
        ok = (ok and positions.shape == rows and positions.dtype is torch.int32 and positions.get_device() == index
              and positions.is_contiguous())
    rot = 0
    if inv_freq is not None:
        rot = 2 * inv_freq.shape[0] if inv_freq.dim() == 1 else -1
        ok = (ok and rot >= 0 and inv_freq.dtype is torch.float32 and inv_freq.get_device() == index
              and inv_freq.is_contiguous())
    if q_weight is not None:
        ok = (ok and norm and q_weight.shape == d and q_weight.dtype is torch.float32 and q_weight.get_device() == index
              and q_weight.is_contiguous())
    if k_weight is not None:
        ok = (ok and norm and k_weight.shape == d and k_weight.dtype is torch.float32 and k_weight.get_device() == index
              and k_weight.is_contiguous())
    if not ok:
        if dt not in _DTYPES:
            raise ValueError("unsupported dtype %s" % dt)
        if not 3 <= len(shape) <= 4:
            raise ValueError("rows must be [B,H,T,d] or [H,T,d] (got shape %s)" % (tuple(shape),))
        like = lambda t: shape[:-3] + t.shape[-3:-2] + shape[-2:] if t.dim() >= 3 else shape
        _explain([(_check_rows, n, t, index, dt, like(t)) for n, t in (("q", q), ("k", k)) if t is not None]
                 + ([(check, "positions", positions, index, torch.int32, rows)] if positions is not None else [])
                 + ([(check, "inv_freq", inv_freq, index, torch.float32, (inv_freq.numel(),))] if inv_freq is not None else [])
                 + _weights(q_weight, k_weight, norm, index, d))
    if not x.is_cuda:
        on_gpu(fn, x)
    return qs, ks, qst, kst, index, rot


def _weights(q_weight, k_weight, norm, index, d):
    out = []
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            out += [(check, name, w, index, torch.float32, d)] if norm else [(_refuse, "%s goes with norm" % name)]
    return out


def _refuse(text):
    raise ValueError(text)


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
    qs, ks, qst, kst, index, rot = _rope_inputs("head_rope_fwd", q, k, inv_freq, positions, q_weight, k_weight, norm)
    for name, o, t in (("q_out", q_out, q), ("k_out", k_out, k)) if q_out is not None or k_out is not None else ():
        if o is not None:
            if t is None:
                raise ValueError("%s goes with %s" % (name, name[0]))
            _check_rows(name, o, index, t.dtype, t.shape)
    with scope(index, stream):
        if q_out is None and qs is not None:
            q_out = torch.empty_like(q)
        if k_out is None and ks is not None:
            k_out = torch.empty_like(k)
        desc = _rope_desc(qs, ks, qst, kst, q_out.stride() if qs is not None else (), k_out.stride() if ks is not None else (),
                          (), (), rot, (q if qs is not None else k).dtype, bool(interleaved), bool(norm), float(eps),
                          float(rope_scale))
        st = (_lib or _library()).kda_head_rope_fwd(
            desc, None if q is None else q.data_ptr(), None if k is None else k.data_ptr(), ptr(q_weight), ptr(k_weight),
            ptr(inv_freq), ptr(positions), None if q is None else q_out.data_ptr(), None if k is None else k_out.data_ptr(),
            raw_stream(index, stream))
    if st:
        _check("kda_head_rope_fwd", st)
    return q_out, k_out


def head_rope_bwd(q, k, inv_freq, dq_out, dk_out, positions=None, *, interleaved=False, rope_scale=1.0, q_weight=None,
                  k_weight=None, norm=True, eps=1e-6, workspace=None, stream=None):
    """Backward of ``head_rope_fwd`` through ``kda_head_rope_bwd``.

    Inputs as the forward's; dq_out, dk_out: gradients of its outputs, in their shape and type, any
    strides. Returns (dq, dk, dq_weight, dk_weight): rows in their input's type, weight gradients [d]
    fp32; None for each input that was not given."""
    qs, ks, qst, kst, index, rot = _rope_inputs("head_rope_bwd", q, k, inv_freq, positions, q_weight, k_weight, norm)
    x = q if qs is not None else k
    dt = x.dtype
    zqs, zks = dq_out.stride() if dq_out is not None else (), dk_out.stride() if dk_out is not None else ()
    if not ((dq_out is None if qs is None else dq_out is not None and dq_out.shape == qs and dq_out.dtype is dt and zqs[-1] == 1
             and dq_out.get_device() == index)
            and (dk_out is None if ks is None else dk_out is not None and dk_out.shape == ks and dk_out.dtype is dt
                 and zks[-1] == 1 and dk_out.get_device() == index)):
        for name, g, t in (("dq_out", dq_out, q), ("dk_out", dk_out, k)):
            if (g is None) != (t is None):
                raise ValueError("%s goes with %s" % (name, name[1]))
            if g is not None:
                _check_rows(name, g, index, dt, t.shape)
    if workspace is not None:
        _check_workspace(workspace, x.device)
    with scope(index, stream):
        dq = dk = dwq = dwk = None
        dqs = dks = ()
        if qs is not None:
            dq = torch.empty_like(q)
            dqs = dq.stride()
            if q_weight is not None:
                dwq = torch.empty_like(q_weight)
        if ks is not None:
            dk = torch.empty_like(k)
            dks = dk.stride()
            if k_weight is not None:
                dwk = torch.empty_like(k_weight)
        desc, need = _rope_bwd_desc(qs, ks, qst, kst, zqs, zks, dqs, dks, rot, dt, bool(interleaved), bool(norm), float(eps),
                                    float(rope_scale))
        if dwq is None and dwk is None:
            need = 0
        workspace = _workspace(need, workspace, x.device)
        st = (_lib or _library()).kda_head_rope_bwd(
            desc, ptr(q), ptr(k), ptr(q_weight), ptr(k_weight), ptr(inv_freq), ptr(positions), ptr(dq_out), ptr(dk_out), ptr(dq),
            ptr(dk), ptr(dwq), ptr(dwk), ptr(workspace), _nbytes(workspace), raw_stream(index, stream))
    if st:
        _check("kda_head_rope_bwd", st)
    return dq, dk, dwq, dwk


def _sequences_ok(index, N, cu_seqlens, kv_lens, block_table):
    """What tells sequences and pages apart: N sequences' lengths and table."""
    return (kv_lens.shape == (N,) and kv_lens.dtype is torch.int32 and kv_lens.get_device() == index
            and kv_lens.is_contiguous() and block_table.dim() == 2 and block_table.shape[0] == N
            and block_table.dtype is torch.int32 and block_table.get_device() == index
            and (block_table.stride(1) == 1 or block_table.shape[1] == 1)
            and (cu_seqlens is None or cu_seqlens.dtype is torch.int32 and cu_seqlens.get_device() == index
                 and cu_seqlens.dim() == 1 and cu_seqlens.is_contiguous()))


def _sequence_checks(index, N, cu_seqlens, kv_lens, block_table):
    return ([(check, "cu_seqlens", cu_seqlens, index, torch.int32, (N + 1,))] if cu_seqlens is not None else []) + [
        (check, "kv_lens", kv_lens, index, torch.int32, (N,)),
        (_check_rows, "block_table", block_table, index, torch.int32, (N, block_table.shape[-1] if block_table.dim() else 0))]


def _rows_dims(t, cu_seqlens):
    """Sequences of [N,H,T,d] rows, or of packed [H,T,d] ones."""
    if t.dim() != (4 if cu_seqlens is None else 3):
        raise ValueError("rows must be [H,T,d] with cu_seqlens, [N,H,T,d] without (got shape %s)" % (tuple(t.shape),))
    return t.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1


@functools.lru_cache(maxsize=1024)
def _append_desc(q, k, v, q_strides, k_strides, v_strides, qo, kc, kcs, vcs, N, max_pages, table_stride, rot, dtype, packed,
                 interleaved, norm, eps, rope_scale):
    return KvAppendDesc(N, q[-3] if q is not None else 0, k[-3], k[-2], k[-1], v[-1], rot, kc[0], kc[2], max_pages,
                        table_stride, *(_strides(s) for s in (q_strides, k_strides, v_strides, qo)),
                        *(PageStrides(*s[:3]) for s in (kcs, vcs)), _DTYPES[dtype], packed, interleaved, norm, eps, rope_scale)


def kv_append(q, k, v, k_cache, v_cache, block_table, kv_lens, inv_freq=None, *, cu_seqlens=None, interleaved=False,
              rope_scale=1.0, q_weight=None, k_weight=None, norm=True, eps=1e-6, q_out=None, stream=None):
    """New tokens' keys and values into a paged cache, through ``kda_kv_append``: k normed and rotated
    at its position on the way, v copied; q (or None) normed and rotated into the returned q_out (bf16).

    q, k, v: [N,Hq,T,dk], [N,Hk,T,dk], [N,Hk,T,dv], T new tokens of each of N sequences, or packed
    [H,T,d] with cu_seqlens (int32 [N+1]); bf16 or fp32, any strides with contiguous channels.
    k_cache, v_cache: [pages,Hk,page_size,dk], [pages,Hk,page_size,dv] bf16, written in place, any
    strides with contiguous channels. block_table: int32 [N,max_pages], or one row expanded to that; position
    j of sequence s is row j % page_size of page block_table[s, j // page_size]. kv_lens: int32 [N], positions in use
    with the new tokens, which are each sequence's last. Norm and rotation as ``head_rope_fwd``."""
    BF16 = torch.bfloat16
    N = _rows_dims(k, cu_seqlens)
    index, dt, ks, kst, vs, vst = k.get_device(), k.dtype, k.shape, k.stride(), v.shape, v.stride()
    kc, kcs, vc, vcs = k_cache.shape, k_cache.stride(), v_cache.shape, v_cache.stride()
    qs, qst = (q.shape, q.stride()) if q is not None else (None, ())
    rot = 0 if inv_freq is None else 2 * inv_freq.shape[0] if inv_freq.dim() == 1 else -1
    d = ks[-1:]
    if not (dt in _DTYPES and v.dtype is dt and k_cache.dtype is BF16 and v_cache.dtype is BF16 and kst[-1] == 1
            and (vst[-1] == 1 or vs[-1] == 1) and vs[:-1] == ks[:-1] and v.get_device() == index and len(kc) == 4 and len(vc) == 4
            and kc[1] == ks[-3] and kc[3:] == d and kc[:3] == vc[:3] and vc[3:] == vs[-1:] and kcs[3] == 1
            and (vcs[3] == 1 or vs[-1] == 1) and k_cache.get_device() == index and v_cache.get_device() == index
            and (q is None or q.dtype is dt and qst[-1] == 1 and len(qs) == len(ks) and qs[:-3] == ks[:-3] and qs[-2:] == ks[-2:]
                 and q.get_device() == index)
            and (inv_freq is None or rot >= 0 and inv_freq.dtype is torch.float32 and inv_freq.get_device() == index
                 and inv_freq.is_contiguous())
            and (q_weight is None or norm and q_weight.shape == d and q_weight.dtype is torch.float32
                 and q_weight.get_device() == index and q_weight.is_contiguous())
            and (k_weight is None or norm and k_weight.shape == d and k_weight.dtype is torch.float32
                 and k_weight.get_device() == index and k_weight.is_contiguous())
            and _sequences_ok(index, N, cu_seqlens, kv_lens, block_table)):
        if dt not in _DTYPES:
            raise ValueError("unsupported dtype %s" % dt)
        if len(kc) != 4:
            raise ValueError("k_cache must be [pages,Hk,page_size,dk] (got shape %s)" % (tuple(kc),))
        like = ks[:-3] + (qs[-3:-2] if qs is not None and len(qs) >= 3 else ks[-3:-2]) + ks[-2:]
        _explain([(_check_rows, "k", k, index, dt, ks), (_check_rows, "v", v, index, dt, ks[:-1] + vs[-1:])]
                 + ([(_check_rows, "q", q, index, dt, like)] if q is not None else [])
                 + [(_check_rows, "k_cache", k_cache, index, BF16, (kc[0], ks[-3], kc[2], ks[-1])),
                    (_check_rows, "v_cache", v_cache, index, BF16, (kc[0], ks[-3], kc[2], vs[-1]))]
                 + ([(check, "inv_freq", inv_freq, index, torch.float32, (inv_freq.numel(),))] if inv_freq is not None else [])
                 + _weights(q_weight, k_weight, norm, index, d) + _sequence_checks(index, N, cu_seqlens, kv_lens, block_table))
    if q_out is not None:
        if q is None:
            raise ValueError("q_out goes with q")
        _check_rows("q_out", q_out, index, BF16, q.shape)
    if not k.is_cuda:
        on_gpu("kv_append", k)
    with scope(index, stream):
        if q_out is None and q is not None:
            q_out = torch.empty_like(q, dtype=BF16)
        desc = _append_desc(qs, ks, vs, qst, kst, vst, q_out.stride() if q is not None else (), kc, kcs, vcs, N,
                            block_table.shape[1], block_table.stride(0), rot, dt, cu_seqlens is not None, bool(interleaved),
                            bool(norm), float(eps), float(rope_scale))
        st = (_lib or _library()).kda_kv_append(
            desc, ptr(q), k.data_ptr(), v.data_ptr(), ptr(q_weight), ptr(k_weight), ptr(inv_freq), ptr(cu_seqlens),
            kv_lens.data_ptr(), block_table.data_ptr(), ptr(q_out), k_cache.data_ptr(), v_cache.data_ptr(),
            raw_stream(index, stream))
    if st:
        _check("kda_kv_append", st)
    return q_out


@functools.lru_cache(maxsize=1024)
def _attn_desc(q, q_strides, o_strides, kc, kcs, vc, vcs, N, max_pages, table_stride, window, packed, scale):
    """The call's descriptor and the workspace it needs."""
    desc = PagedAttnDesc(N, q[-3], vc[1], q[-2], q[-1], vc[3], vc[0], vc[2], max_pages, table_stride, window,
                         _strides(q_strides), _strides(o_strides), PageStrides(*kcs[:3]), PageStrides(*vcs[:3]), packed,
                         q[-1] ** -0.5 if scale is None else scale)
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
    A token that sees nothing has o = 0 and lse = -inf; one that sees scores of -inf alone NaN and -inf."""
    BF16 = torch.bfloat16
    N = _rows_dims(q, cu_seqlens)
    index, qs, qst = q.get_device(), q.shape, q.stride()
    kc, kcs, vc, vcs = k_cache.shape, k_cache.stride(), v_cache.shape, v_cache.stride()
    if not (q.dtype is BF16 and k_cache.dtype is BF16 and v_cache.dtype is BF16 and qst[-1] == 1 and len(kc) == 4
            and len(vc) == 4 and kc[:3] == vc[:3] and kc[3:] == qs[-1:] and kcs[3] == 1 and vcs[3] == 1
            and k_cache.get_device() == index and v_cache.get_device() == index
            and _sequences_ok(index, N, cu_seqlens, kv_lens, block_table)):
        if len(kc) != 4 or len(vc) != 4:
            raise ValueError("k_cache and v_cache must be [pages,Hk,page_size,d] (got shapes %s, %s)" % (tuple(kc), tuple(vc)))
        _explain([(_check_rows, "q", q, index, BF16, qs), (_check_rows, "k_cache", k_cache, index, BF16, vc[:3] + qs[-1:]),
                  (_check_rows, "v_cache", v_cache, index, BF16, vc)]
                 + _sequence_checks(index, N, cu_seqlens, kv_lens, block_table))
    out = qs[:-1] + vc[3:]
    if o is not None:
        _check_rows("o", o, index, BF16, out)
    if lse is not None:
        check("lse", lse, index, torch.float32, qs[:-1])
    if workspace is not None:
        _check_workspace(workspace, q.device)
    if not q.is_cuda:
        on_gpu("paged_attn", q)
    with scope(index, stream):
        if o is None:
            if out == qs:
                o = torch.empty_like(q)
            else:      # q's order of dimensions: token-major rows stay so
                turned = qst[-3] < qst[-2]
                o = torch.empty(out[:-3] + (out[-2], out[-3], out[-1]) if turned else out, dtype=BF16, device=q.device)
                o = o.transpose(-3, -2) if turned else o
        if lse is None and return_lse:
            lse = torch.empty(qs[:-1], dtype=torch.float32, device=q.device)
        desc, need = _attn_desc(qs, qst, o.stride(), kc, kcs, vc, vcs, N, block_table.shape[1], block_table.stride(0), int(window),
                                cu_seqlens is not None, None if scale is None else float(scale))
        workspace = _workspace(need, workspace, q.device)
        st = (_lib or _library()).kda_paged_attn(
            desc, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), ptr(cu_seqlens), kv_lens.data_ptr(),
            block_table.data_ptr(), o.data_ptr(), ptr(lse), ptr(workspace), _nbytes(workspace), raw_stream(index, stream))
    if st:
        _check("kda_paged_attn", st)
    return (o, lse) if return_lse else o
