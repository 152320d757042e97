"""Norms around a block with its gate, residual and residual scale (``include/kda_norm.h``).

    block_norm_fwd(f, x=None, ...) -> (x_out, n)      post-norm, gate, residual, next pre-norm
    block_norm_bwd(f, x, dx_out, dn, ...)             gradients of every input
        -> (df, dx, dgate, dnorm_weight, dscale_weight, dpre_weight)
"""
import ctypes
import functools

import torch

from . import _DTYPES, _check, _check_workspace, _nbytes, _workspace, library
from ._launch import check, on_gpu, ptr, raw_stream, scope

NORM_MAX_D = 16384   # KDA_NORM_MAX_D of include/kda_norm.h


class NormDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("D", ctypes.c_int64), ("in_dtype", ctypes.c_int32),
                ("res_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("post_norm", ctypes.c_int32),
                ("pre_norm", ctypes.c_int32), ("scale", ctypes.c_float), ("eps", ctypes.c_float),
                ("pre_eps", ctypes.c_float)]


_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = library()
        P, D, Z, I = ctypes.c_void_p, ctypes.POINTER(NormDesc), ctypes.c_size_t, ctypes.c_int32
        lib.kda_block_norm_fwd.argtypes = [D] + [P] * 9
        lib.kda_block_norm_fwd.restype = I
        lib.kda_block_norm_bwd_workspace_bytes.argtypes = [D]
        lib.kda_block_norm_bwd_workspace_bytes.restype = Z
        lib.kda_block_norm_bwd.argtypes = [D] + [P] * 15 + [Z, P]
        lib.kda_block_norm_bwd.restype = I
        _lib = lib
    return _lib


@functools.lru_cache(maxsize=1024)
def _desc(rows, D, in_dtype, res_dtype, out_dtype, post_norm, pre_norm, scale, eps, pre_eps):
    """The call's descriptor: nothing but its arguments, so calls of one shape share it."""
    return NormDesc(rows, D, _DTYPES[in_dtype], _DTYPES[res_dtype], _DTYPES[out_dtype], post_norm, pre_norm, scale, eps,
                    pre_eps)


def _inputs(f, index, shape, x, gate, norm_weight, post_norm, scale_weight, pre_norm, pre_weight):
    """Checks the inputs both directions share; returns (rows, D)."""
    if f.dtype not in _DTYPES:
        raise ValueError("unsupported input dtype %s" % f.dtype)
    if not shape:
        raise ValueError("f must have at least one dimension")
    D = shape[-1]
    check("f", f, index, f.dtype, shape)
    if x is not None:
        if x.dtype not in _DTYPES:
            raise ValueError("unsupported residual dtype %s" % x.dtype)
        check("x", x, index, x.dtype, shape)
    if gate is not None:
        check("gate", gate, index, f.dtype, shape)
    if norm_weight is not None:
        if not post_norm:
            raise ValueError("norm_weight goes with post_norm")
        check("norm_weight", norm_weight, index, torch.float32, (D,))
    if scale_weight is not None:
        check("scale_weight", scale_weight, index, torch.float32, (D,))
    if pre_weight is not None:
        if not pre_norm:
            raise ValueError("pre_weight goes with pre_norm")
        check("pre_weight", pre_weight, index, torch.float32, (D,))
    return (f.numel() // D if D else 0), D


def block_norm_fwd(f, x=None, *, gate=None, norm_weight=None, post_norm=True, eps=1e-6, scale=1.0, scale_weight=None,
                   pre_norm=True, pre_weight=None, pre_eps=1e-6, res_dtype=None, out_dtype=None, x_out=None, n=None,
                   store_x=True, stream=None):
    """Post-norm, gate, residual and the next pre-norm through ``kda_block_norm_fwd``.

    f: [..., D] bf16 or fp32, the block's output; x: the residual stream, f's shape (bf16 or fp32),
    or None; gate: f's shape and type, or None; weights [D] fp32, or None (ones).
        u = sigmoid(gate) * norm_weight * f / sqrt(mean(f^2) + eps)     (post_norm False: f itself)
        x_out = x + scale * scale_weight * u
        n = pre_weight * x_out / sqrt(mean(x_out^2) + pre_eps)
    Returns (x_out, n): x_out in x's type (``res_dtype``, default f's type, without x), None with
    ``store_x=False``; n in ``out_dtype`` (default f's type), None with ``pre_norm=False``.
    ``x_out=x`` updates the residual stream in place. The sums of a row's squares must be finite in
    fp32. Caller-supplied outputs are checked like the inputs; the others are allocated on
    ``stream``."""
    dev, index, shape = f.device, f.get_device(), f.shape
    rows, D = _inputs(f, index, shape, x, gate, norm_weight, post_norm, scale_weight, pre_norm, pre_weight)
    res_dtype = x.dtype if x is not None else (res_dtype or (x_out.dtype if x_out is not None else f.dtype))
    out_dtype = out_dtype or (n.dtype if n is not None else f.dtype)
    if res_dtype not in _DTYPES or out_dtype not in _DTYPES:
        raise ValueError("unsupported output dtype %s" % (out_dtype if res_dtype in _DTYPES else res_dtype))
    if x_out is not None:
        check("x_out", x_out, index, res_dtype, shape)
    if n is not None:
        if not pre_norm:
            raise ValueError("n goes with pre_norm")
        check("n", n, index, out_dtype, shape)
    if not pre_norm and x_out is None and not store_x:
        raise ValueError("nothing to compute: neither x_out nor n is wanted")
    on_gpu("block_norm_fwd", f)
    desc = _desc(rows, D, f.dtype, res_dtype, out_dtype, bool(post_norm), bool(pre_norm), float(scale), float(eps),
                 float(pre_eps))
    with scope(index, stream):
        if x_out is None and store_x:
            x_out = torch.empty_like(f, dtype=res_dtype)
        if n is None and pre_norm:
            n = torch.empty_like(f, dtype=out_dtype)
        st = (_lib or _library()).kda_block_norm_fwd(desc, ptr(f), ptr(gate), ptr(x), ptr(norm_weight),
                                           ptr(scale_weight), ptr(pre_weight), ptr(x_out), ptr(n),
                                           raw_stream(index, stream))
    _check("kda_block_norm_fwd", st)
    return x_out, n


def block_norm_bwd(f, x, dx_out, dn, *, gate=None, norm_weight=None, post_norm=True, eps=1e-6, scale=1.0,
                   scale_weight=None, pre_norm=True, pre_weight=None, pre_eps=1e-6, dx=None, workspace=None,
                   stream=None):
    """Backward of ``block_norm_fwd`` through ``kda_block_norm_bwd``.

    Inputs as the forward (x as it was before an in-place forward); dx_out: gradient of x_out (x's
    type, or bf16 / fp32 without x), or None; dn: gradient of n (bf16 or fp32), or None.
    Returns (df, dx, dgate, dnorm_weight, dscale_weight, dpre_weight): tensors in their input's
    type, weight gradients [D] fp32; None for each input that was not given. ``dx=dx_out`` updates
    the residual stream's gradient in place."""
    dev, index, shape = f.device, f.get_device(), f.shape
    rows, D = _inputs(f, index, shape, x, gate, norm_weight, post_norm, scale_weight, pre_norm, pre_weight)
    if dx_out is None and dn is None:
        raise ValueError("one of dx_out and dn is required")
    res_dtype = x.dtype if x is not None else (dx_out.dtype if dx_out is not None else f.dtype)
    out_dtype = dn.dtype if dn is not None else f.dtype
    for dt in (res_dtype, out_dtype):
        if dt not in _DTYPES:
            raise ValueError("unsupported gradient dtype %s" % dt)
    if dx_out is not None:
        check("dx_out", dx_out, index, res_dtype, shape)
    if dn is not None:
        if not pre_norm:
            raise ValueError("dn goes with pre_norm")
        check("dn", dn, index, out_dtype, shape)
    if dx is not None:
        if x is None:
            raise ValueError("dx goes with x")
        check("dx", dx, index, res_dtype, shape)
    if workspace is not None:
        _check_workspace(workspace, dev)
    on_gpu("block_norm_bwd", f)
    desc = _desc(rows, D, f.dtype, res_dtype, out_dtype, bool(post_norm), bool(pre_norm), float(scale), float(eps),
                 float(pre_eps))
    lib = _lib or _library()
    sums = norm_weight is not None or scale_weight is not None or pre_weight is not None
    need = lib.kda_block_norm_bwd_workspace_bytes(desc) if sums else 0
    with scope(index, stream):
        df = torch.empty_like(f)
        dgate = torch.empty_like(f) if gate is not None else None
        if dx is None and x is not None:
            dx = torch.empty_like(x)
        dws = [torch.empty_like(w) if w is not None else None for w in (norm_weight, scale_weight, pre_weight)]
        workspace = _workspace(need, workspace, dev)
        st = lib.kda_block_norm_bwd(desc, ptr(f), ptr(gate), ptr(x), ptr(norm_weight),
                                    ptr(scale_weight), ptr(pre_weight), ptr(dx_out), ptr(dn),
                                    ptr(df), ptr(dgate), ptr(dx), *map(ptr, dws),
                                    ptr(workspace), _nbytes(workspace), raw_stream(index, stream))
    _check("kda_block_norm_bwd", st)
    return (df, dx, dgate, *dws)
