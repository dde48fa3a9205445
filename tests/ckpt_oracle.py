"""The 8-bit block format, the norm and the GELU in 64-bit numpy (test infrastructure; shares no code with the
HIP path)."""
import math

import numpy as np
from scipy.special import erfc

INT8, E4M3 = 2, 3
U32 = 2.0 ** -24     # half a step of fp32, relative
U16 = 2.0 ** -8      # of bf16


def e4m3_table():
    """The 256 values of the e4m3 codes: 4 exponent bits (bias 7), 3 fraction bits, no infinities, 0x7F NaN."""
    t = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = (1 + f / 8) * 2.0 ** (e - 7) if e else f * 2.0 ** -9
        if e == 15 and f == 7:
            v = math.nan
        t[c] = -v if c & 128 else v
    return t


_TAB = e4m3_table()


def pack(x, fmt):
    """(codes [rows, 32 nb], exponent bytes [rows, nb]) of fp32 x [rows, n], computed exactly."""
    rows, n = x.shape
    nb = -(-n // 32)
    b = np.zeros((rows, nb * 32))
    b[:, :n] = x.astype(np.float64)
    b = b.reshape(rows, nb, 32)
    amax = np.abs(b).max(-1)
    bad = ~np.isfinite(b).all(-1)
    top = 127.0 if fmt == INT8 else 448.0
    s = np.ones((rows, nb), np.int64)
    for r in range(rows):
        for k in range(nb):
            if bad[r, k]:
                s[r, k] = 255
                continue
            m, e = math.frexp(amax[r, k] / top)        # amax <= top 2^(s - 127), s smallest
            s[r, k] = 1 if amax[r, k] == 0 else max(1, (e - 1 if m == 0.5 else e) + 127)
    sc = np.where(bad, 1.0, np.exp2(s.astype(np.float64) - 127))[..., None]
    with np.errstate(invalid="ignore"):
        v = np.where(bad[..., None], 0.0, b) / sc
    if fmt == INT8:
        q = np.rint(v).astype(np.int64) & 255
    else:
        a = np.abs(v)
        pos = _TAB[:127]                                 # ascending codes 0..126
        hi = np.clip(np.searchsorted(pos, a, "left"), 0, 126)
        lo = np.maximum(hi - 1, 0)
        dl, dh = a - pos[lo], pos[hi] - a
        c = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
        c = np.where(pos[hi] == a, hi, c)
        q = c | np.where(np.signbit(v), 128, 0)
        q = np.where(bad[..., None], 0, q)
    return q.astype(np.uint8).reshape(rows, nb * 32), s.astype(np.uint8)


def unpack(q, s, fmt, n):
    rows, nb = s.shape
    v = q.astype(np.int8).astype(np.float64) if fmt == INT8 else _TAB[q]
    sc = np.where(s == 255, np.inf, np.exp2(s.astype(np.float64) - 127))
    with np.errstate(invalid="ignore"):
        return (v.reshape(rows, nb, 32) * sc[..., None]).reshape(rows, nb * 32)[:, :n]


def norm_fwd(h, gain, eps):
    h = h.astype(np.float64)
    rstd = 1 / np.sqrt((h * h).mean(-1) + eps)
    return h * rstd[:, None] * gain.astype(np.float64), rstd


def norm_bwd(h, gain, rstd, dy, dr):
    """(dx, dgain) and the sums of the magnitudes of their terms."""
    h, gain, r, dy = (np.asarray(a, np.float64) for a in (h, gain, rstd, dy))
    r = r[:, None]
    xh, w = h * r, dy * gain
    dx = r * (w - xh * (w * xh).mean(-1, keepdims=True))
    ax = r * (np.abs(w) + np.abs(xh) * np.abs(w * xh).mean(-1, keepdims=True))
    if dr is not None:
        dx, ax = dx + dr, ax + np.abs(dr)
    return dx, (dy * xh).sum(0), ax, np.abs(dy * xh).sum(0)


def phi_cdf(x):
    return 0.5 * erfc(-np.asarray(x, np.float64) / math.sqrt(2))


def gelu(x):
    return np.asarray(x, np.float64) * phi_cdf(x)


def gelu_slope(x):
    x = np.asarray(x, np.float64)
    return phi_cdf(x) + x * np.exp(-x * x / 2) / math.sqrt(2 * math.pi)
