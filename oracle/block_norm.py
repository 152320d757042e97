"""fp64 norms around a block with gate, residual and residual scale, their backward, and bounds on
what fp32 may lose.

The bounds are running error bounds: an fp32 evaluation of an expression is off by at most K U32
times the same expression with every term's magnitude, K the number of roundings on its longest
path. A row's sum has at most 16 terms a thread, 6 shuffles and 16 waves (38), squares and products
one more, the root and reciprocal 2 each, a sigmoid 6 + |v|.
"""
import numpy as np

from .glr import U32, sigmoid

K_SUM = 42.0


def evaluate(f, x, gate, w_post, lam, w_pre, *, post, pre, scale, eps, pre_eps, dxo=None, dn=None):
    """dict of the outputs (and, with dxo or dn, gradients), each with its bound under '<name>_b'."""
    c64 = lambda t: None if t is None else np.asarray(t, np.float64)
    f, x, gate, w_post, lam, w_pre, dxo, dn = map(c64, (f, x, gate, w_post, lam, w_pre, dxo, dn))
    D = f.shape[-1]
    one = np.ones(D)
    wp, lm, wr = (one if t is None else t for t in (w_post, lam, w_pre))
    mean = lambda t: t.mean(-1, keepdims=True)
    r1 = 1.0 / np.sqrt(mean(f * f) + eps) if post else np.ones(f.shape[:-1] + (1,))
    k1 = K_SUM / 2 + 4 if post else 0.0                # relative error of r1, in U32
    fh = f * r1
    p = fh * wp
    s = sigmoid(gate) if gate is not None else np.ones_like(f)
    ks = 6.0 + np.abs(gate) if gate is not None else 0.0
    u = p * s
    ku = k1 + ks + 4.0
    add = scale * lm * u
    xo = add + (x if x is not None else 0.0)
    xo_b = U32 * ((ku + 3.0) * np.abs(add) + np.abs(xo))
    out = {"x_out": xo, "x_out_b": xo_b}
    if pre:
        ms = mean(xo * xo) + pre_eps
        r2 = 1.0 / np.sqrt(ms)
        # the error of the mean square is twice sum |x'| err(x'), half of it passes to its root
        k2 = K_SUM / 2 + 4 + mean(np.abs(xo) * xo_b) / ms / U32
        xh = xo * r2
        xh_b = r2 * xo_b + U32 * (k2 + 1.0) * np.abs(xh)
        out["n"], out["n_b"] = xh * wr, np.abs(wr) * (xh_b + U32 * np.abs(xh))
    if dxo is None and dn is None:
        return out
    d = dxo if dxo is not None else np.zeros_like(f)
    d_b = np.zeros_like(f)
    d_m = np.abs(d)
    if dn is not None:
        t = dn * wr
        m2 = mean(t * xh)
        m2_b = mean(np.abs(t) * xh_b) + U32 * K_SUM * mean(np.abs(t * xh))
        out["dw_pre"] = (dn * xh).reshape(-1, D).sum(0)
        out["dw_pre_b"] = _sum_bound(np.abs(dn) * xh_b, np.abs(dn * xh))
        inner = np.abs(t) + np.abs(xh) * (np.abs(m2))
        d = d + r2 * (t - xh * m2)
        d_b = r2 * (U32 * (k2 + 6.0) * inner + np.abs(m2) * xh_b + np.abs(xh) * m2_b) + U32 * (d_m + r2 * inner)
        d_m = d_m + r2 * inner
    out["dx"], out["dx_b"] = d, d_b
    out["dlam"] = scale * (d * u).reshape(-1, D).sum(0)
    out["dlam_b"] = abs(scale) * _sum_bound(np.abs(u) * d_b + U32 * (ku + 2.0) * np.abs(u) * d_m, np.abs(u) * d_m)
    sl = np.abs(scale * lm)
    du, du_b, du_m = d * scale * lm, sl * (d_b + 2.0 * U32 * d_m), sl * d_m
    out["dgate"] = du * p * s * (1.0 - s)
    # 1 - s is formed from s: an absolute error of s's own
    out["dgate_b"] = (np.abs(p) * s * (1.0 - s) * (du_b + U32 * (ku + 6.0) * du_m)
                      + U32 * (ks * s + 1.0) * du_m * np.abs(p) * s)
    dp, dp_b, dp_m = du * s, s * (du_b + U32 * (ks + 1.0) * du_m), s * du_m
    if post:
        out["dw_post"] = (dp * fh).reshape(-1, D).sum(0)
        out["dw_post_b"] = _sum_bound(np.abs(fh) * (dp_b + U32 * (k1 + 2.0) * dp_m), np.abs(fh) * dp_m)
        t1, t1_b, t1_m = dp * wp, np.abs(wp) * (dp_b + U32 * dp_m), np.abs(wp) * dp_m
        m1 = mean(t1 * fh)
        m1_b = mean(np.abs(fh) * (t1_b + U32 * (k1 + K_SUM) * t1_m))
        df = r1 * (t1 - fh * m1)
        out["df_b"] = r1 * (t1_b + np.abs(fh) * m1_b + U32 * (2.0 * k1 + 6.0) * (t1_m + np.abs(fh * m1)))
        out["df"] = df
    else:
        out["df"], out["df_b"] = dp, dp_b
    return out


def _sum_bound(err, mag):
    """Bound on a column sum: the terms' errors, and one rounding per addition on the longest path
    (rows of a workgroup, its row groups, the workgroups: never more than the rows)."""
    D = mag.shape[-1]
    rows = mag.reshape(-1, D).shape[0]
    return err.reshape(-1, D).sum(0) + U32 * (rows + 2.0) * mag.reshape(-1, D).sum(0)
