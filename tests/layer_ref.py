"""Plain 64-bit reference of the layer operators (numpy), with error bounds of the binary32
arithmetic between the inputs and a result's one rounding.  Written from the definitions; shares
no code with the library or the oracle."""
import numpy as np
from scipy.special import ndtr

U = 2.0 ** -24                       # half a step of binary32, relative
HALF = {"bf16": 2.0 ** -8, "f32": U}  # of a stored result
GROUP = 32


def code_values(fmt):
    """value of each of the 256 code bytes (NaN where there is none)"""
    v = np.empty(256)
    for c in range(256):
        if fmt == "int8":
            v[c] = c - 256 if c >= 128 else c
            continue
        e, m = (c >> 3) & 15, c & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if (e, m) == (15, 7) else -x if c & 128 else x
    return v


def ckpt(x, fmt):
    """(values, scale bytes) of the checkpoint of x (float64, R x C): for every group the smallest
    allowed power of two, found by trying them, and for every element the nearest code, the even
    one of two as near."""
    R, C = x.shape
    n = -(-C // GROUP)
    pad = np.zeros((R, n * GROUP))
    pad[:, :C] = x
    g = pad.reshape(R * n, GROUP)
    with np.errstate(invalid="ignore"):
        big = np.abs(g).max(1)
    finite = np.isfinite(g).all(1)
    low, top = (-124, 464.0) if fmt == "e4m3" else (-127, 127.5)
    s = np.full(R * n, low)
    for k in range(low, 128):
        lim = top * 2.0 ** k
        s = np.where((big > lim) if fmt == "e4m3" else (big >= lim), k + 1, s)
    vals = code_values(fmt)
    pos = np.unique(np.abs(vals[~np.isnan(vals)]))       # 0 = the even code, then in code order
    if fmt == "int8":
        pos = pos[pos <= 127]
    v = np.abs(np.where(finite[:, None], g, 0.0)) / 2.0 ** s[:, None].astype(float)
    i = np.clip(np.searchsorted(pos, v), 1, len(pos) - 1)
    lo, hi = pos[i - 1], pos[i]
    pick_hi = (hi - v < v - lo) | ((hi - v == v - lo) & (i % 2 == 0))
    q = np.where(pick_hi, hi, lo) * np.sign(g) * 2.0 ** s[:, None].astype(float)
    q = np.where(finite[:, None], q, np.nan)
    byte = np.where(finite, s + 127, 255).astype(np.uint8)
    return q.reshape(R, n * GROUP)[:, :C], byte.reshape(R, n)


def norm(x, w, b, kind, eps, dtype):
    """y, mean, rstd and the bounds of their errors.  m roundings bound a sum of C terms however
    it is ordered inside a lane (C / 64 terms) and across lanes (a tree)."""
    C = x.shape[1]
    m = 16 + C / 64
    mean = x.mean(1, keepdims=True) if kind == "layer" else np.zeros((x.shape[0], 1))
    d = x - mean
    var = (d * d).mean(1, keepdims=True)
    rstd = 1 / np.sqrt(var + eps)
    dmean = m * U * np.abs(x).mean(1, keepdims=True) if kind == "layer" else 0 * mean
    # var: (m + 4) roundings of its terms, the mean's own error (squared, for their cross term
    # vanishes) and the part of it that its rounding adds to every difference
    dvar = (m + 4) * U * var + dmean * dmean
    rrel = np.minimum(0.5 * dvar / (var + eps) + 4 * U, 1.0)
    bias = 0 if b is None else b
    y = d * rstd * w + bias
    ey = (np.abs(w) * rstd * dmean * (1 + rrel) + np.abs(d * rstd * w) * (rrel + 4 * U)
          + 2 * U * (np.abs(y) + np.abs(bias)))
    ey = ey + (np.abs(y) + ey) * HALF[dtype]
    return dict(y=y, mean=mean[:, 0], rstd=rstd[:, 0], ey=ey, emean=dmean[:, 0] + U * np.abs(mean[:, 0]),
                erstd=rrel[:, 0] * rstd[:, 0])


def norm_grads(dy, x, w, b, mean, rstd, kind, dtype, dres=None):
    """dx, dw, db, y and bounds, for given statistics (float64 copies of the binary32 ones)."""
    R, C = x.shape
    m = 16 + C / 64
    mean = mean[:, None] if kind == "layer" else np.zeros((R, 1))
    rstd = rstd[:, None]
    xh = (x - mean) * rstd                        # binary32: 2 roundings
    g = dy * w
    c1 = g.mean(1, keepdims=True) if kind == "layer" else 0 * mean
    c2 = (g * xh).mean(1, keepdims=True)
    dx = rstd * (g - c1 - xh * c2)
    e = rstd * U * ((m + 2) * (np.abs(g).mean(1, keepdims=True) + np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True))
                    + 6 * (np.abs(g) + np.abs(c1) + np.abs(xh * c2)))
    if dres is not None:
        dx = dx + dres
        e = e + U * np.abs(dx)
    edx = e + (np.abs(dx) + e) * HALF[dtype]
    # R terms in any order: R - 1 roundings of partial sums, and 4 of each term
    edw = (R + 4) * U * np.abs(dy * xh).sum(0)
    edb = R * U * np.abs(dy).sum(0)
    bias = 0 if b is None else b
    y = xh * w + bias
    ey = 4 * U * np.abs(xh * w) + U * (np.abs(y) + np.abs(bias))
    ey = ey + (np.abs(y) + ey) * HALF[dtype]
    return dict(dx=dx, dw=(dy * xh).sum(0), db=dy.sum(0), y=y, edx=edx, edw=edw, edb=edb, ey=ey)


def act(h, kind):
    """f(h), f'(h)"""
    h = np.asarray(h, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "relu":
            return np.where(h > 0, h, 0 * h), np.where(h > 0, 1.0, 0.0)
        if kind == "silu":
            s = 1 / (1 + np.exp(-h))
            return h * s, s * (1 + h * (1 - s))
        if kind == "gelu":
            return h * ndtr(h), ndtr(h) + h * np.exp(-h * h / 2) / np.sqrt(2 * np.pi)
        a, c = np.sqrt(2 / np.pi), 0.044715
        t = np.tanh(a * (h + c * h ** 3))
        return h * (1 + t) / 2, (1 + t) / 2 + h / 2 * (1 - t * t) * a * (1 + 3 * c * h * h)


def act_bounds(h, kind):
    """Bounds of the binary32 errors of f(h) and f'(h).  The logistic function s(z) of an argument
    z with relative error r has the relative error (1 - s) |z| r; z and e^z together take 8
    roundings and a hardware exponential and reciprocal of 1 step each, so r |z| <= 8 U |z| and a
    further 6 U.  |z| (1 - s) s <= 0.28 and |h| stays in units of the result: both functions are
    within 16 U of |h| + 1, and of 4 U relative for large h.  Phi is within 1e-7 absolutely."""
    h = np.abs(np.asarray(h, np.float64))
    if kind == "relu":
        return 0 * h, 0 * h
    if kind == "gelu":
        return (1e-7 + 8 * U) * h, 1e-7 + 16 * U + 8 * U * h * np.exp(-h * h / 2) * (1 + h * h)
    return 16 * U * h, 32 * U + 0 * h
