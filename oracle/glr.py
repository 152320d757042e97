"""fp64 gated linear recurrence, token by token, with its reverse and bounds on what fp32 may lose.

    h_t = a_t h_{t-1} + w(a_t) i_t x_t,  a = exp(la),  la given or g_min sigmoid(e^A z)

Arrays are [rows, channels] for one sequence of one head. ``sequences`` cuts a batch in either
layout into them.
"""
import numpy as np

U32 = 2.0 ** -24   # half a step of fp32


def sigmoid(x):
    x = np.asarray(x, np.float64)
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def gates(x, la=None, z=None, A=None, g_min=-5.0, u=None, scale="one"):
    """dict of every gate quantity of one sequence (float64)."""
    x = np.asarray(x, np.float64)
    q = {"x": x}
    if z is not None:
        z, A = np.asarray(z, np.float64), np.asarray(A, np.float64)
        q["z"], q["eA"] = z, np.exp(A)
        q["s"] = sigmoid(q["eA"] * z)
        q["la"] = g_min * q["s"]
    else:
        q["la"] = np.asarray(la, np.float64)
    q["a"] = np.exp(q["la"])
    one_minus = -np.expm1(q["la"])
    if scale == "one":
        q["w"], q["dw"] = np.ones_like(x), np.zeros_like(x)
    elif scale == "leaky":
        q["w"], q["dw"] = one_minus, -q["a"]
    else:
        q["w"] = np.sqrt(-np.expm1(2.0 * q["la"]))
        with np.errstate(divide="ignore", invalid="ignore"):
            q["dw"] = np.where(q["w"] > 0, -q["a"] ** 2 / q["w"], 0.0)
    q["u"] = None if u is None else np.asarray(u, np.float64)
    q["i"] = np.ones_like(x) if u is None else sigmoid(u)
    return q


def forward(q, S0):
    """(h [rows, C], states before each row [rows, C], last state)."""
    x = q["x"]
    b = q["w"] * q["i"] * x
    h = np.array(S0, np.float64)
    hs, prev = np.empty_like(x), np.empty_like(x)
    for t in range(x.shape[0]):
        prev[t] = h
        h = q["a"][t] * h + b[t]
        hs[t] = h
    return hs, prev, h


def backward(q, prev, dy, dS_T, g_min=-5.0):
    """dict of the gradients of one sequence (dA summed over its rows)."""
    g = np.array(dS_T, np.float64)
    G = np.empty_like(q["x"])
    for t in range(G.shape[0] - 1, -1, -1):
        G[t] = dy[t] + g
        g = q["a"][t] * G[t]
    i, w, x = q["i"], q["w"], q["x"]
    r = {"G": G, "dS0": g, "dx": G * w * i, "du": G * w * x * i * (1.0 - i)}
    r["dla"] = G * (q["a"] * prev + q["dw"] * i * x)
    if "z" in q:
        slope = g_min * q["eA"] * q["s"] * (1.0 - q["s"])
        r["dd"] = r["dla"] * slope
        r["dA"] = (r["dd"] * q["z"]).sum(0)
    else:
        r["dd"] = r["dla"]
    return r


# ---- what fp32 may lose -----------------------------------------------------------------------
# Every fp32 operation is off by at most U32 of its result, the exponential, reciprocal and square
# root of the hardware by at most 2 U32. Counting them along each path:
#   sigmoid(v)      exponent's argument |v| U32, exp 3, sum 1, reciprocal 2: (6 + |v|) U32
#   la from z       e^A 3, e^A z 1 (an absolute error 4 |e^A z| of sigmoid's argument), sigmoid, g_min: ra U32
#   a               exp 3 and its argument |la|, and la's error |la| ra
#   w               1 - a: the series 4 + ra, or past -0.35 the difference, a / (1 - a) <= 2.4 times a's error;
#                   the root of it adds 1 + a, product and root
# The recurrence adds one rounding a step, and a split over chunks at most doubles each count (the
# products of decays are formed once more, in another order).

def _counts(q, scale):
    ra = 8.0 + 5.0 * np.abs(q["eA"] * q["z"]) if "z" in q else np.zeros_like(q["x"])
    with np.errstate(invalid="ignore"):
        ca = 3.0 + np.where(np.isinf(q["la"]), 0.0, np.abs(q["la"]) * (1.0 + ra))
    cw = np.zeros_like(ca) if scale == "one" else 6.0 + ra + 2.4 * ca
    if scale == "norm":
        cw = cw + ca + 4.0
    ci = np.zeros_like(ca) if q["u"] is None else 6.0 + np.minimum(np.abs(q["u"]), 200.0)
    return ra, ca, cw, ci


def forward_bound(q, S0, scale):
    """(bound on |h error| per row, bound on the last state's)."""
    _, ca, cw, ci = _counts(q, scale)
    b = np.abs(q["w"] * q["i"] * q["x"])
    H, E = np.abs(np.array(S0, np.float64)), np.zeros(q["x"].shape[1:])
    out = np.empty_like(q["x"])
    for t in range(out.shape[0]):
        aH = q["a"][t] * H
        H = aH + b[t]
        E = q["a"][t] * E + 2.0 * U32 * ((ca[t] + 1.0) * aH + (cw[t] + ci[t] + 3.0) * b[t] + H)
        out[t] = E
    return out, E


def backward_bounds(q, prev, hbound, dy, dS_T, scale, S0, g_min=-5.0):
    """Bounds on the errors of dx, du, dd, dA and dS0, given the forward's bound per row."""
    ra, ca, cw, ci = _counts(q, scale)
    T = q["x"].shape[0]
    ag, E = np.abs(np.array(dS_T, np.float64)), np.zeros(q["x"].shape[1:])
    GA, GE = np.empty_like(q["x"]), np.empty_like(q["x"])
    for t in range(T - 1, -1, -1):
        GA[t] = np.abs(dy[t]) + ag
        GE[t] = E + 2.0 * U32 * GA[t]
        ag = q["a"][t] * GA[t]
        E = q["a"][t] * GE[t] + 2.0 * U32 * (ca[t] + 1.0) * ag
    w, i, x = np.abs(q["w"]), q["i"], np.abs(q["x"])
    r = {"dS0": E}
    r["dx"] = GE * w * i + U32 * (cw + ci + 3.0) * GA * w * i
    # 1 - i is formed from i: an absolute error of i's own error, which stays under ci + 1 of 1
    r["du"] = (GE * w * i * (1.0 - i) + U32 * (cw + ci + 6.0) * GA * w * i * (1.0 - i)
               + U32 * (ci * i + 1.0) * GA * w * i) * x
    pe = np.zeros_like(hbound)
    pe[1:] = hbound[:-1]
    dw = np.abs(q["dw"])
    mag = q["a"] * np.abs(prev) + dw * i * x
    err = q["a"] * pe + U32 * ((ca + 2.0) * q["a"] * np.abs(prev) + (2.0 * ca + cw + ci + 6.0) * dw * i * x)
    dla = GE * mag + GA * (err + 2.0 * U32 * mag)
    if "z" in q:
        slope = np.abs(g_min * q["eA"] * q["s"] * (1.0 - q["s"]))
        # 1 - s: s's error is ra of s
        e = dla * slope + U32 * (2.0 * ra + 8.0) * GA * mag * slope + U32 * (ra * q["s"] + 1.0) * GA * mag * np.abs(
            g_min * q["eA"] * q["s"])
        r["dd"] = e
        m = GA * mag * slope * np.abs(q["z"])
        # a thread adds at most 256 rows, then the partial sums of its chunks and sequences
        r["dA"] = (e * np.abs(q["z"])).sum(0) + U32 * (512.0 + T / 64.0) * m.sum(0)
    else:
        r["dd"] = dla
    return r


def sequences(N, H, T, cu=None):
    """(n, h, index of the sequence's rows in x) of every (sequence, head) of a batch."""
    for n in range(N):
        for h in range(H):
            if cu is None:
                yield n, h, (n, h, slice(0, T))
            else:
                yield n, h, (h, slice(int(cu[n]), int(cu[n + 1])))
