"""Gated linear recurrence (``include/kda_glr.h``): h_t = alpha_t h_{t-1} + w(alpha_t) i_t x_t per
(sequence, head, channel), with its backward and its single-token step.

    glr_fwd(x, log_alpha, S0=None, ...) -> (y, S_T, entry_states)    prefill, fixed or packed
    glr_bwd(x, log_alpha, S0, dy, dS_T=None, ...)                     gradients of every input
        -> (dx, ddecay, din_gate, dS0, dA_log)
    glr_step(x, log_alpha, S, ...) -> y                               one token, S updated in place
"""
import ctypes
import functools

import torch

from . import _DTYPES, _check, _check_workspace, _nbytes, _workspace, library
from ._launch import check, on_gpu, ptr, raw_stream, scope

GLR_CHUNK = 128   # KDA_GLR_CHUNK of include/kda_glr.h
_SCALES = {"one": 0, "leaky": 1, "norm": 2}


class GlrDesc(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("H", ctypes.c_int64), ("T", ctypes.c_int64), ("d", ctypes.c_int64),
                ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("packed", ctypes.c_int32),
                ("scale", ctypes.c_int32), ("g_min", ctypes.c_float)]


class GlrGates(ctypes.Structure):
    _fields_ = [("log_alpha", ctypes.c_void_p), ("z", ctypes.c_void_p), ("A_log", ctypes.c_void_p),
                ("in_gate", ctypes.c_void_p)]


_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = library()
        P, D, G, Z, I = (ctypes.c_void_p, ctypes.POINTER(GlrDesc), ctypes.POINTER(GlrGates), ctypes.c_size_t,
                         ctypes.c_int32)
        lib.kda_glr_fwd_workspace_bytes.argtypes = [D]
        lib.kda_glr_fwd_workspace_bytes.restype = Z
        lib.kda_glr_fwd.argtypes = [D, P, G, P, P, P, P, P, P, Z, P]
        lib.kda_glr_fwd.restype = I
        lib.kda_glr_bwd_workspace_bytes.argtypes = [D, I, I]
        lib.kda_glr_bwd_workspace_bytes.restype = Z
        lib.kda_glr_bwd.argtypes = [D, P, G] + [P] * 11 + [Z, P]
        lib.kda_glr_bwd.restype = I
        lib.kda_glr_step.argtypes = [D, P, G, P, P, P]
        lib.kda_glr_step.restype = I
        _lib = lib
    return _lib


def _scale(input_scale):
    try:
        return _SCALES[input_scale]
    except KeyError:
        raise ValueError("input_scale must be one of %s (got %r)" % (sorted(_SCALES), input_scale)) from None


def _gates(x, index, shape, log_alpha, z, A_log, in_gate, H, d):
    """Checked gates of a call: exactly one of log_alpha and z, A_log [H,d] fp32 with z."""
    dt = x.dtype
    if z is None:
        if log_alpha is None:
            raise ValueError("give exactly one of log_alpha and z")
        if A_log is not None:
            raise ValueError("A_log goes with z")
        check("log_alpha", log_alpha, index, dt, shape)
        decay = (log_alpha.data_ptr(), None, None)
    else:
        if log_alpha is not None:
            raise ValueError("give exactly one of log_alpha and z")
        if A_log is None:
            raise ValueError("A_log goes with z")
        check("z", z, index, dt, shape)
        check("A_log", A_log, index, torch.float32, (H, d))
        decay = (None, z.data_ptr(), A_log.data_ptr())
    if in_gate is None:
        return GlrGates(*decay, None)
    check("in_gate", in_gate, index, dt, shape)
    return GlrGates(*decay, in_gate.data_ptr())


def _dtype(x, out_dtype):
    if x.dtype not in _DTYPES:
        raise ValueError("unsupported input dtype %s" % x.dtype)
    out_dtype = out_dtype or x.dtype
    if out_dtype not in _DTYPES:
        raise ValueError("unsupported output dtype %s" % out_dtype)
    return out_dtype


@functools.lru_cache(maxsize=1024)
def _desc(N, H, T, d, in_dtype, out_dtype, packed, input_scale, g_min):
    """The call's descriptor: nothing but its arguments, so calls of one shape share it."""
    return GlrDesc(N, H, T, d, _DTYPES[in_dtype], _DTYPES[out_dtype], packed, _scale(input_scale), g_min)


def _batch(x, cu_seqlens):
    """(N, H, T, d) of a fixed [N,H,T,d] or packed [H,T,d] batch."""
    if cu_seqlens is None:
        if x.dim() != 4:
            raise ValueError("x must be [N,H,T,d] without cu_seqlens (got %s)" % (tuple(x.shape),))
        return tuple(x.shape)
    if x.dim() != 3:
        raise ValueError("x must be [H,T,d] with cu_seqlens (got %s)" % (tuple(x.shape),))
    check("cu_seqlens", cu_seqlens, x.get_device(), torch.int32, (cu_seqlens.numel(),))
    N = cu_seqlens.numel() - 1
    if N < 1:
        raise ValueError("cu_seqlens must have at least 2 entries")
    return (N,) + tuple(x.shape)


def _entry_shape(N, H, T, d, packed):
    return (H if packed else N * H, -(-T // GLR_CHUNK), d)


def glr_fwd(x, log_alpha=None, S0=None, *, z=None, A_log=None, g_min=-5.0, in_gate=None, input_scale="one",
            cu_seqlens=None, out_dtype=None, y=None, S_T=None, store_state=True, entry_states=None,
            store_entry_states=False, workspace=None, stream=None):
    """Prefill of the gated linear recurrence through ``kda_glr_fwd``.

    x: [N,H,T,d], or packed [H,T,d] with ``cu_seqlens`` (int32 [N+1] on the device); bf16 or fp32.
    The decay is ``log_alpha`` (x's shape and type, <= 0) or g_min * sigmoid(exp(A_log) * z) from
    ``z`` (x's shape and type) and ``A_log`` [H,d] fp32. With ``in_gate`` (x's shape and type), x is
    multiplied by sigmoid(in_gate); ``input_scale`` is "one", "leaky" (1 - alpha) or "norm"
    (sqrt(1 - alpha^2)). S0, S_T: [N,H,d] fp32 (S_T may be S0).
    Returns (y, S_T, entry_states): y of x's shape; S_T None with ``store_state=False``;
    entry_states (the states kda_glr_bwd restarts from) None unless ``store_entry_states`` or a
    tensor for them is given. Packed rows in no sequence are left as they are in y (a y that the
    call allocates holds nothing meaningful there).
    Caller-supplied outputs and workspace are checked like the inputs; what the call allocates is
    allocated on ``stream`` (default: the current stream of x's device).
    """
    out_dtype = _dtype(x, out_dtype)
    dev, index, shape = x.device, x.get_device(), x.shape
    N, H, T, d = _batch(x, cu_seqlens)
    packed = cu_seqlens is not None
    check("x", x, index, x.dtype, shape)
    gates = _gates(x, index, shape, log_alpha, z, A_log, in_gate, H, d)
    for name, t in (("S0", S0), ("S_T", S_T)):
        if t is not None:
            check(name, t, index, torch.float32, (N, H, d))
    if y is not None:
        check("y", y, index, out_dtype, shape)
    eshape = _entry_shape(N, H, T, d, packed)
    if entry_states is not None:
        check("entry_states", entry_states, index, torch.float32, eshape)
    if workspace is not None:
        _check_workspace(workspace, dev)
    on_gpu("glr_fwd", x)
    desc = _desc(N, H, T, d, x.dtype, out_dtype, packed, input_scale, float(g_min))
    lib = _lib or _library()
    need = lib.kda_glr_fwd_workspace_bytes(desc)
    with scope(index, stream):
        if y is None:
            y = torch.empty_like(x, dtype=out_dtype)
        if S_T is None and store_state:
            S_T = torch.empty(N, H, d, device=dev, dtype=torch.float32)
        if entry_states is None and store_entry_states:
            entry_states = torch.empty(eshape, device=dev, dtype=torch.float32)
        workspace = _workspace(need, workspace, dev)
        st = lib.kda_glr_fwd(desc, ptr(x), gates, ptr(cu_seqlens), ptr(S0), ptr(y), ptr(S_T),
                             ptr(entry_states), ptr(workspace), _nbytes(workspace), raw_stream(index, stream))
    _check("kda_glr_fwd", st)
    return y, S_T, entry_states


def glr_bwd(x, log_alpha, S0, dy, dS_T=None, *, z=None, A_log=None, g_min=-5.0, in_gate=None, input_scale="one",
            cu_seqlens=None, entry_states=None, workspace=None, stream=None):
    """Backward of ``glr_fwd`` through ``kda_glr_bwd``.

    Inputs as ``glr_fwd``; dy: x's shape, bf16 or fp32 (the forward's output type); dS_T: [N,H,d]
    fp32 or None; ``entry_states``: what the forward stored for the same inputs (without them the
    call recomputes them). Returns (dx, ddecay, din_gate, dS0, dA_log): dx, ddecay (the gradient of
    log_alpha, or of z) and din_gate (None without in_gate) in x's shape and type, dS0 [N,H,d] fp32,
    dA_log [H,d] fp32 (None without z). Packed rows in no sequence are left unwritten in the
    gradients."""
    _dtype(x, dy.dtype)
    dev, index, shape = x.device, x.get_device(), x.shape
    N, H, T, d = _batch(x, cu_seqlens)
    packed = cu_seqlens is not None
    check("x", x, index, x.dtype, shape)
    gates = _gates(x, index, shape, log_alpha, z, A_log, in_gate, H, d)
    check("dy", dy, index, dy.dtype, shape)
    for name, t in (("S0", S0), ("dS_T", dS_T)):
        if t is not None:
            check(name, t, index, torch.float32, (N, H, d))
    if entry_states is not None:
        check("entry_states", entry_states, index, torch.float32, _entry_shape(N, H, T, d, packed))
    if workspace is not None:
        _check_workspace(workspace, dev)
    on_gpu("glr_bwd", x)
    desc = _desc(N, H, T, d, x.dtype, dy.dtype, packed, input_scale, float(g_min))
    lib = _lib or _library()
    need = lib.kda_glr_bwd_workspace_bytes(desc, entry_states is not None, z is not None)
    with scope(index, stream):
        dx, dd = torch.empty_like(x), torch.empty_like(x)
        du = torch.empty_like(x) if in_gate is not None else None
        dA = torch.empty(H, d, device=dev, dtype=torch.float32) if z is not None else None
        dS0 = torch.empty(N, H, d, device=dev, dtype=torch.float32)
        workspace = _workspace(need, workspace, dev)
        st = lib.kda_glr_bwd(desc, ptr(x), gates, ptr(cu_seqlens), ptr(S0), ptr(entry_states),
                             ptr(dy), ptr(dS_T), ptr(dx), ptr(dd), ptr(du), ptr(dA),
                             ptr(dS0), ptr(workspace), _nbytes(workspace), raw_stream(index, stream))
    _check("kda_glr_bwd", st)
    return dx, dd, du, dS0, dA


def glr_step(x, log_alpha, S, *, z=None, A_log=None, g_min=-5.0, in_gate=None, input_scale="one", out_dtype=None,
             y=None, stream=None):
    """One token of the gated linear recurrence through ``kda_glr_step``; S ([N,H,d] fp32) is
    updated in place. x and the gates: [N,H,d] as a token of ``glr_fwd``. Returns y [N,H,d]."""
    out_dtype = _dtype(x, out_dtype)
    index, shape = x.get_device(), x.shape
    if len(shape) != 3:
        raise ValueError("x must be [N,H,d] (got %s)" % (tuple(shape),))
    N, H, d = shape
    check("x", x, index, x.dtype, shape)
    gates = _gates(x, index, shape, log_alpha, z, A_log, in_gate, H, d)
    check("S", S, index, torch.float32, shape)
    if y is not None:
        check("y", y, index, out_dtype, shape)
    on_gpu("glr_step", x)
    desc = _desc(N, H, 1, d, x.dtype, out_dtype, False, input_scale, float(g_min))
    with scope(index, stream):
        if y is None:
            y = torch.empty_like(x, dtype=out_dtype)
        st = (_lib or _library()).kda_glr_step(desc, x.data_ptr(), gates, S.data_ptr(), y.data_ptr(),
                                               raw_stream(index, stream))
    _check("kda_glr_step", st)
    return y
