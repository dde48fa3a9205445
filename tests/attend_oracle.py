"""Norms and rotation of queries and keys, the cache's formats and the attention over it in 64-bit numpy (test
infrastructure; shares no code with the HIP path)."""
import math

import numpy as np

from tests import ckpt_oracle as O

INT8, E4M3, E2M1 = 2, 3, 4
HALF, PAIRS = 0, 1
E2M1_VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def grid(x, fmt):
    """What a cache keeps of fp32 x [..., d], as the values it stands for (exact)."""
    shape = x.shape
    rows = x.reshape(-1, shape[-1])
    if fmt != E2M1:
        return O.unpack(*O.pack(rows, fmt), fmt, shape[-1]).reshape(shape)
    n, d = rows.shape
    nb = -(-d // 32)
    b = np.zeros((n, nb * 32))
    b[:, :d] = rows.astype(np.float64)
    b = b.reshape(n, nb, 32)
    bad = ~np.isfinite(b).all(-1)
    amax = np.where(bad, 0.0, np.abs(np.where(np.isfinite(b), b, 0.0)).max(-1))
    s = np.ones((n, nb), np.int64)
    for r in range(n):
        for k in range(nb):
            if amax[r, k] > 0:
                m, e = math.frexp(amax[r, k] / 6.0)      # amax <= 6 2^(s - 127), s smallest
                s[r, k] = max(1, (e - 1 if m == 0.5 else e) + 127)
    sc = np.exp2(s.astype(np.float64) - 127)[..., None]
    v = np.where(bad[..., None], 0.0, b) / sc
    a = np.abs(v)
    hi = np.clip(np.searchsorted(E2M1_VALUES, a, "left"), 0, 7)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - E2M1_VALUES[lo], E2M1_VALUES[hi] - a
    c = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    out = np.where(np.signbit(v), -1.0, 1.0) * E2M1_VALUES[c] * sc
    out = np.where(bad[..., None], np.nan, out)
    return out.reshape(n, nb * 32)[:, :d].reshape(shape)


def frequencies(rot, base, factor=1.0, trained=0.0, low=1.0, high=32.0):
    f = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    w = np.zeros_like(f)
    if trained > 0:
        w = np.clip((trained * f / (2 * math.pi) - low) / (high - low), 0, 1)
    return f * (w + (1 - w) / factor)


def table(positions, rot, base=10000.0, amplitude=1.0, **scaled):
    """cos | sin, 64 bits [positions, rot]."""
    a = np.arange(positions, dtype=np.float64)[:, None] * frequencies(rot, base, **scaled)
    return np.concatenate([np.cos(a), np.sin(a)], -1) * amplitude


def rotate(y, tab, pos, layout, back=False):
    """(rotated y [t, h, d], sum of its terms' magnitudes)."""
    r = tab.shape[-1] // 2
    c, s = tab[pos][:, None, :r].astype(np.float64), tab[pos][:, None, r:].astype(np.float64)
    if back:
        s = -s
    first, second = (slice(0, r), slice(r, 2 * r)) if layout == HALF else (slice(0, 2 * r, 2), slice(1, 2 * r, 2))
    out, mag = y.copy(), np.abs(y)
    a, b = y[..., first], y[..., second]
    out[..., first], out[..., second] = a * c - b * s, b * c + a * s
    mag[..., first] = np.abs(a * c) + np.abs(b * s)
    mag[..., second] = np.abs(b * c) + np.abs(a * s)
    return out, mag


def qk_fwd(x, gain, eps, tab=None, pos=None, layout=HALF):
    y = x.astype(np.float64)
    if gain is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * gain.astype(np.float64)
    return y if tab is None else rotate(y, tab, pos, layout)[0]


def qk_bwd(x, dy, gain, eps, tab=None, pos=None, layout=HALF):
    """(dx, dgain, and the sums of the magnitudes of their terms)."""
    x, dy = x.astype(np.float64), dy.astype(np.float64)
    mag = np.abs(dy)
    if tab is not None:
        dy, mag = rotate(dy, tab, pos, layout, back=True)
    if gain is None:
        return dy, None, mag, None
    g = gain.astype(np.float64)
    rstd = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh, w, mw = x * rstd, dy * g, mag * np.abs(g)
    dx = rstd * (w - xh * (w * xh).mean(-1, keepdims=True))
    ax = rstd * (mw + np.abs(xh) * (mw * np.abs(xh)).mean(-1, keepdims=True))
    return dx, (dy * xh).sum((0, 1)), ax, (mag * np.abs(xh)).sum((0, 1))


def attend(q, k, v, scale, limits):
    """One sequence: q [n, hq, d], k and v [len, hk, d]; query i sees tokens 0..limits[i].  (out, Sum p |v|, the largest
    sum of a score's terms' magnitudes a row sees, the largest |score|), the last two [n, hq]."""
    n, hq, d = q.shape
    hk = k.shape[1]
    out, mag = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    terms, top = np.zeros((n, hq)), np.zeros((n, hq))
    q = q.astype(np.float64)
    for i in range(n):
        m = int(limits[i]) + 1
        if m <= 0:
            continue
        for h in range(hq):
            c = h // (hq // hk)
            s = scale * (k[:m, c] @ q[i, h])
            with np.errstate(invalid="ignore"):
                p = np.exp(s - s.max())
                p /= p.sum()
            out[i, h], mag[i, h] = p @ v[:m, c], p @ np.abs(v[:m, c])
            terms[i, h] = scale * (np.abs(k[:m, c]) @ np.abs(q[i, h])).max()
            top[i, h] = np.abs(s).max()
    return out, mag, terms, top


def attend_tol(n, d, mag, terms, top, kept=0.0):
    """How far the output may be off over n tokens.  A score is a sum of 3 d products' parts, each addition off by at
    most a step (2 u); its exponent is rounded twice (the scale, the fused product and offset) and the exponential by a
    step: a probability's relative error, with what it is rounded to (kept).  Probabilities and values are added up in at
    most n / 8 + 64 steps of 2 u each, numerator and denominator; then the quotient and the output's rounding."""
    u = O.U32
    nb = -(-d // 32)
    p = 3 * 32 * nb * 2 * u * terms + 3 * u * (top + terms) * 1.5 + 4 * u + kept
    return np.expm1(2 * p + 2 * (n / 8 + 64) * 2 * u + 4 * u)[..., None] * mag
