"""Plain 64-bit references of rotary positions, token log probabilities and 8-bit AdamW states (numpy), with
bounds of the binary32 arithmetic between the inputs and a result's one rounding.  Written from the
definitions; shares no code with the library or the oracle."""
import numpy as np

U = 2.0 ** -24                        # half a step of binary32, relative
HALF = {"bf16": 2.0 ** -8, "f32": U}  # of a stored result
LOG2E, LN2 = 1 / np.log(2.0), np.log(2.0)


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def freqs(rot, base=10000.0, scaling="none", factor=1.0, trained_len=0, low=1.0, high=32.0):
    i = np.arange(rot // 2, dtype=np.longdouble)
    if scaling == "ntk":
        base = np.longdouble(base) * np.longdouble(factor) ** (np.longdouble(rot) / (rot - 2))
    f = np.longdouble(base) ** (-2 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":
        k = np.clip((trained_len * f / (2 * np.pi) - low) / (high - low), 0, 1)
        f = f * k + f / factor * (1 - k)
    return f.astype(np.float64)


def rotary(x, f, pos, layout, scale, sign, dtype):
    """(value, bound) of x [B, T, H, D] (float64 copies) rotated; f: the frequencies given, pos: [B, T].
    The library's angle in turns takes three roundings of binary64 and one of binary32 of at most half a
    turn (2^-26 of a turn), its sine and cosine are within 4 U; the products and their difference take
    three roundings more."""
    n = len(f)
    w = pos.astype(np.longdouble)[:, :, None] * f.astype(np.longdouble)
    c, s = np.cos(w).astype(float)[:, :, None], sign * np.sin(w).astype(float)[:, :, None]
    off = (2 * np.pi * 2.0 ** -26 + 4 * U + np.abs(w).astype(float) * 2.0 ** -51)[:, :, None]
    a, b = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    y, e = x.copy(), np.zeros_like(x)
    y[..., a] = scale * (x[..., a] * c - x[..., b] * s)
    y[..., b] = scale * (x[..., a] * s + x[..., b] * c)
    size = abs(scale) * (np.abs(x[..., a]) + np.abs(x[..., b])) * (off + 4 * U)
    for i in (a, b):
        e[..., i] = size + (np.abs(y[..., i]) + size) * HALF[dtype] + 2.0 ** -133
    return y, e


# ---------------------------------------------------------------------------
# log probabilities
# ---------------------------------------------------------------------------
def joins(cols):
    """Bound of the joins of partial sums that a term passes: one for every 2048 columns, and 32 across
    lanes, waves and parts of a row."""
    return 32 + cols / 2048


def logprob(x, tokens, scale):
    """Statistics and log probabilities of rows x (float64, R x C), with bounds.  A term's exponent u (in
    powers of two) takes a difference, a rounded constant and a product: 3 |u| U ln 2 <= 2.1 |u| U, and
    moves between maxima add as much again in all; the hardware's exponential 2 U; every join 3 roundings."""
    R, C = x.shape
    with np.errstate(all="ignore"):
        z = x * scale
        top32 = (x.max(1).astype(np.float32) * np.float32(scale)).astype(np.float64)
        top = z.max(1)
        empty = np.isneginf(top32) & ~np.isnan(x).any(1)
        bad = np.isnan(x).any(1) | np.isposinf(x).any(1) | np.isposinf(top32)
        safe = np.where(empty | bad, 0.0, top)
        d = np.where((empty | bad)[:, None], -np.inf, z - safe[:, None])
        e = np.exp(d)
        s = np.where(empty | bad, 1.0, e.sum(1))
        p = e / s[:, None]
        u = np.where(e > 0, np.abs(d), 0.0) * LOG2E
        # never through max + log s, which loses the sum beside masks of the type's lowest value
        logsum = np.log(s) + (safe - np.where(empty | bad, 0.0, top32))
        pu = (p * u).sum(1)
        puu = (p * u * u).sum(1)
        J = joins(C)
        ds = (4.2 * pu + 2 + 8 + 3 * J) * U
        elogsum = ds + 4 * U * (1 + np.abs(logsum) + np.log(s))
        H = np.log(s) + LN2 * pu
        eH = LN2 * U * (4.2 * puu + (12 + 4 * J) * pu) + ds * (1 + LN2 * pu) + 4 * U * (1 + np.log(s) + pu)
        lp = (z - safe[:, None]) - np.log(s)[:, None]
        elp = elogsum[:, None] + 2 * U * (np.abs(z - np.where(empty | bad, 0.0, top32)[:, None]) + np.abs(lp))
    # a log probability that binary32 cannot hold rounds to -infinity
    lp[lp < -float(np.finfo(np.float32).max) * (1 + U / 2)] = -np.inf
    lp[empty] = -np.inf
    lp[bad] = np.nan
    H[empty], logsum[empty], p[empty] = 0.0, 0.0, 0.0
    H[bad], logsum[bad], p[bad] = np.nan, np.nan, np.nan
    top32 = np.where(np.isnan(x).any(1), np.where(np.isnan(x), -np.inf, x).max(1).astype(np.float32) * np.float32(scale), top32)
    valid = (tokens >= 0) & (tokens < C)
    at = np.where(valid, tokens, 0)
    rows = np.arange(R)
    elp = np.where(np.isfinite(elp), elp, 0.0)
    return dict(max=top32, logsum=logsum, elogsum=elogsum, entropy=H, eentropy=eH, lp=lp, elp=elp, p=p, empty=empty,
                logprob=np.where(valid, lp[rows, at], 0.0), elogprob=np.where(valid, elp[rows, at], 0.0))


def top(x, k):
    """Columns of the k largest logits, in falling order, equal ones by rising column; NaN as -infinity."""
    v = np.where(np.isnan(x), -np.inf, x) + 0.0
    return np.argsort(-v, axis=1, kind="stable")[:, :k]


def logprob_grad(x, tokens, dl, dh, mx, logsum, H, scale, dtype):
    """Gradient of the logits (and bounds) for given statistics: -log p takes 3 roundings of terms as large as
    the difference from the maximum and the logarithm of the sum; the exponential of it 2 U."""
    R, C = x.shape
    valid = (tokens >= 0) & (tokens < C)
    dl = np.where(valid, dl, 0.0)
    zero = ((dl == 0) & (dh == 0)) | (np.isneginf(mx) & (logsum == 0))
    with np.errstate(all="ignore"):
        d = x * scale - mx[:, None]
        lp = d - logsum[:, None]
        p = np.exp(lp)
        size = np.where(np.isneginf(d), 0.0, np.abs(d)) + np.abs(logsum)[:, None]
        rel = (4 * size + 8) * U
        hot = np.zeros_like(x)
        hot[np.flatnonzero(valid), tokens[valid]] = 1.0
        w = np.where(p > 0, p * (np.where(np.isneginf(lp), 0.0, lp) + H[:, None]), p)
        dz = dl[:, None] * (hot - p) - np.where(dh == 0, 0.0, dh)[:, None] * w
        part = np.abs(dl)[:, None] * p + np.abs(dh)[:, None] * p * (np.where(np.isneginf(lp), 0.0, np.abs(lp)) + np.abs(H)[:, None])
        e = scale * (part * (rel + 6 * U) + np.abs(dh)[:, None] * p * size * 4 * U + 3 * U * (part + np.abs(dl)[:, None] * hot))
        y = scale * dz
        e = e + (np.abs(y) + e) * HALF[dtype] + 2.0 ** -126 * scale * (np.abs(dl) + np.abs(dh) * 200)[:, None] + 2.0 ** -133
    y[zero] = 0.0
    e[zero] = 0.0
    return y, e


# ---------------------------------------------------------------------------
# AdamW with 8-bit states
# ---------------------------------------------------------------------------
M_VALUES = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127])
V_VALUES = np.array([m * 2.0 ** -17 if e == 0 else (8 + m) * 2.0 ** (e - 18) for e in range(31) for m in range(8)])


def scales_at(n):
    return -(-n // 16) * 16


def state_bytes(n):
    return scales_at(n) + -(-n // 32)


def read_state(buf, n, which):
    """Values (float64) that an 8-bit state stands for."""
    codes, byte = buf[:n].astype(int), buf[scales_at(n):state_bytes(n)].astype(int)
    if which == "m":
        v = np.where(codes % 128 == 127, np.nan, np.concatenate([M_VALUES, [0]])[codes % 128]) * np.where(codes >= 128, -1, 1)
    else:
        v = np.where(codes > 247, np.nan, np.concatenate([V_VALUES, np.zeros(8)])[codes])
    scale = np.where(byte == 255, np.nan, np.where(byte == 0, 0.0, 2.0 ** (byte - 127.0)))
    return v * np.repeat(scale, 32)[:n]


def key(seed, step, tensor):
    low = (1 << 64) - 1

    def mix(k):
        k &= low
        k = ((k ^ (k >> 30)) * 0xBF58476D1CE4E5B9) & low
        k = ((k ^ (k >> 27)) * 0x94D049BB133111EB) & low
        return k ^ (k >> 31)

    golden = 0x9E3779B97F4A7C15
    return mix(mix(seed + golden * step) + golden * (tensor + 1)) & 0xFFFFFFFF


def random16(n, k, first=0):
    """(for m, for v) of elements first .. first + n"""
    j = np.arange(first, first + n, dtype=np.uint64)
    x = ((j & 0xFFFFFFFF) * 0x9E3779B1 + k + (j >> 32) * 0xDDB3D743) & 0xFFFFFFFF
    x ^= x >> 15
    x = (x * 0xB504F333) & 0xFFFFFFFF
    x ^= x >> 13
    x = (x * 0xDDB3D743) & 0xFFFFFFFF
    x ^= x >> 16
    return x >> 16, x & 0xFFFF


def write_state(x, r, which):
    """The 8-bit state of binary32 values x with 16-bit random numbers r: the smallest allowed scale, found by
    trying them; then steps of an eighth of the power of two below a value, rounded down after adding the
    random part of a step (in binary32, as the sum is defined)."""
    values, low, emin = (M_VALUES, -124, -6) if which == "m" else (V_VALUES, -116, -14)
    n = len(x)
    buf = np.zeros(state_bytes(n), np.uint8)
    pad = np.zeros(-(-n // 32) * 32)
    pad[:n] = np.abs(x)
    g = pad.reshape(-1, 32)
    finite = np.isfinite(g).all(1)
    big = np.where(finite, g.max(1), 0.0)
    s = np.full(len(g), low)
    for e in range(low, 128):
        s = np.where(big > values[-1] * 2.0 ** e, e + 1, s)
    buf[scales_at(n):] = np.where(finite, s + 127, 255)
    y = (np.where(finite[:, None], g, 0.0) * 2.0 ** -s[:, None].astype(float)).reshape(-1)[:n]
    e = np.maximum(np.floor(np.log2(np.where(y > 0, y, 1e-300))), emin)
    e = np.where(2.0 ** e > y, np.maximum(e - 1, emin), e)          # the logarithm is rounded
    e = np.where(2.0 ** (e + 1) <= y, e + 1, e)
    k = np.floor((y * 2.0 ** (3 - e)).astype(np.float32) + r.astype(np.float32) * np.float32(2.0 ** -16)).astype(float)
    code = np.searchsorted(values, k * 2.0 ** (e - 3))
    assert np.array_equal(values[code], k * 2.0 ** (e - 3))
    buf[:n] = code + (128 if which == "m" else 0) * np.signbit(x) if which == "m" else code
    buf[:n] *= np.repeat(finite, 32)[:n]
    return buf


def adam_f32(p, g, m, v, cfg, gs=None):
    """One AdamW step, every operation rounded to binary32, and how far a step with 8-bit states may take p from
    it.  That step's square root, 1 / bc2 and 1 / den are off by 2 U, U and 2 U, its products by U each (three) and
    its sum by U: 9 U of the update; here the root, two quotients, a product and the sum are off by U each: 5 U.
    The last differences round both results, by U of them each; products below 2^-126 may be flushed."""
    f = np.float32
    lr, (b1, b2), eps, wd, t = cfg["lr"], cfg.get("betas", (0.9, 0.999)), cfg.get("eps", 1e-8), cfg.get("weight_decay", 0.0), cfg["step"]
    decay, step_size, bc2 = f(1 - lr * wd), f(lr / (1 - b1 ** t)), f(np.sqrt(1 - b2 ** t))
    with np.errstate(all="ignore"):
        g = g if gs is None else g * f(gs)
        p = p * decay
        m = f(b1) * m + f(1 - b1) * g
        v = f(b2) * v + f(1 - b2) * (g * g)
        update = step_size * (m / (np.sqrt(v) / bc2 + f(eps)))
        p = p - update
        off = 14 * U * np.abs(update.astype(float)) + 2 * U * np.abs(p.astype(float)) + 2.0 ** -126
    return p, m, v, off
