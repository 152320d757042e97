"""fp64 head norms with rotation, their backward, the append to a paged cache and the attention over it,
with bounds on what the kernels' fp32 (and the probabilities' bf16) may lose.

Bounds count roundings, U32 = 2^-24 each, against the terms' magnitudes:
  * a row's sum of squares: 16 fma a lane and 6 shuffled additions, the mean and eps 3 more; its root
    halves that, root and reciprocal 1 each, two products: K_Y = 20 relative on y, 18 on x / rms;
  * cos and sin: the reduced angle is at most pi/4 and rounded once, the series add at most 3 roundings
    of values up to 1: 4 absolute, the scale 1 more, products and sum 3: K_R = 8 on |a| + |b|.
"""
import numpy as np

from .glr import U32

K_Y, K_R, K_SUM = 20.0, 8.0, 24.0
U16 = 2.0 ** -8                      # half a step of bf16, relative


def pairs(d, rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def angles(positions, inv_freq):
    return np.asarray(positions, np.float64)[..., None] * np.asarray(inv_freq, np.float32).astype(np.float64)


def rotate(y, th, rot, interleaved, scale, sign=1.0):
    """Pairs of y's first rot channels turned by sign * th, times scale; th broadcasts over y's rows."""
    z = np.array(y, np.float64)
    if rot:
        a, b = pairs(y.shape[-1], rot, interleaved)
        c, s = np.cos(th) * scale, sign * np.sin(th) * scale
        z[..., a], z[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    return z


def _spread(m, rot, interleaved, scale):
    """|a| + |b| at both members of a pair, times scale; other channels as they are."""
    out = np.array(m, np.float64)
    if rot:
        a, b = pairs(m.shape[-1], rot, interleaved)
        out[..., a] = out[..., b] = (m[..., a] + m[..., b]) * abs(scale)
    return out


def head_rope(x, w, th, *, rot, interleaved, scale, norm, eps, dz=None):
    """x [..., d], th [..., rot/2] -> dict of z (and dx, dw for the gradient dz of z), each with '<name>_b'."""
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    w = np.ones(d) if w is None else np.asarray(w, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps) if norm else np.ones(x.shape[:-1] + (1,))
    xh = x * r
    y = xh * w if norm else x
    ky = K_Y if norm else 0.0
    out = {"z": rotate(y, th, rot, interleaved, scale),
           "z_b": U32 * (ky + K_R) * _spread(np.abs(y), rot, interleaved, scale)}
    if dz is None:
        return out
    dz = np.asarray(dz, np.float64)
    dy = rotate(dz, th, rot, interleaved, scale, -1.0)
    dy_m = _spread(np.abs(dz), rot, interleaved, scale)
    dy_b = U32 * K_R * dy_m
    if not norm:
        out["dx"], out["dx_b"] = dy, dy_b
        return out
    xh_b = U32 * K_Y * np.abs(xh)
    t, t_b = dy * w, np.abs(w) * (dy_b + U32 * np.abs(dy))
    m = (t * xh).mean(-1, keepdims=True)
    m_b = (np.abs(xh) * t_b + np.abs(t) * xh_b).mean(-1, keepdims=True) + U32 * K_SUM * np.abs(t * xh).mean(-1, keepdims=True)
    out["dx"] = r * (t - xh * m)
    out["dx_b"] = r * (t_b + np.abs(m) * xh_b + np.abs(xh) * m_b + U32 * (K_Y + 3.0) * (np.abs(t) + np.abs(xh * m)))
    rows = dy.size // d
    out["dw"] = (dy * xh).reshape(-1, d).sum(0)
    out["dw_b"] = ((np.abs(xh) * dy_b + np.abs(dy) * xh_b).reshape(-1, d).sum(0)
                   + U32 * (rows + 2.0) * np.abs(dy * xh).reshape(-1, d).sum(0))
    return out


def places(cu, kv_lens, table, page_size, pages):
    """For every packed row: (sequence, position, page, row in it); page -1 where it is not stored, sequence -1
    where the row is in none."""
    out = []
    N = len(kv_lens)
    for t in range(int(cu[-1])):
        s = int(np.searchsorted(np.asarray(cu[1:]), t, side="right")) if t >= cu[0] else -1
        if s < 0:
            out.append((-1, 0, -1, 0))
            continue
        assert s < N
        pos = int(kv_lens[s]) - (int(cu[s + 1]) - int(cu[s])) + t - int(cu[s])
        page = -1
        if 0 <= pos < len(table[s]) * page_size:
            page = int(table[s][pos // page_size])
            page = page if 0 <= page < pages else -1
        out.append((s, pos, page, pos % page_size))
    return out


def paged_attn(q, k_cache, v_cache, table, kv_lens, cu, *, scale, window=0):
    """q [T,Hq,dk] packed -> o [T,Hq,dv], o_b, lse [T,Hq], lse_b: token by token, in fp64.

    The scores' products of bf16 numbers are exact in fp32, their sum rounds at most dk times and its
    scaling twice, the exponential 3 times and by the rounded argument's size: e. The probabilities
    enter the second product in bf16 (U16) and their sum in fp32, one rounding a key at most."""
    q = np.asarray(q, np.float64)
    T, Hq, dk = q.shape
    Hk, page_size, dv = v_cache.shape[1], v_cache.shape[2], v_cache.shape[3]
    G = Hq // Hk
    o, o_b = np.zeros((T, Hq, dv)), np.zeros((T, Hq, dv))
    lse, lse_b = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for s in range(len(kv_lens)):
        n, kv = int(cu[s + 1]) - int(cu[s]), int(kv_lens[s])
        if n == 0:
            continue
        pg = [int(p) for p in table[s][:-(-kv // page_size)]]
        K = np.asarray(k_cache[pg], np.float64).transpose(1, 0, 2, 3).reshape(Hk, -1, dk)[:, :kv]
        V = np.asarray(v_cache[pg], np.float64).transpose(1, 0, 2, 3).reshape(Hk, -1, dv)[:, :kv]
        for i in range(n):
            pos = kv - n + i
            lo = max(0, pos - window + 1) if window else 0
            if pos < 0 or lo > pos:
                continue
            t = int(cu[s]) + i
            for h in range(Hq):
                Kh, Vh = K[h // G, lo:pos + 1], V[h // G, lo:pos + 1]
                x = Kh @ q[t, h] * scale
                e = U32 * (dk + 4.0) * (np.abs(Kh) @ np.abs(q[t, h])) * abs(scale)
                m = x.max()
                p = np.exp(x - m)
                l = p.sum()
                lse[t, h] = m + np.log(l)
                err = e + U32 * (4.0 + 3.0 * np.abs(x - m) + 2.0 * abs(m))
                l_rel = (p * err).sum() / l + U32 * (len(p) + 8.0)
                lse_b[t, h] = l_rel + U32 * 4.0 * (abs(m) + np.log(l) + 1.0)
                pr = p / l
                o[t, h] = pr @ Vh
                o_b[t, h] = (pr * (U16 + err + l_rel + U32 * (len(p) + 8.0))) @ np.abs(Vh)
    return o, o_b, lse, lse_b
