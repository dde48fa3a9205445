"""The residual norm at its numeric borders: the roundings that the 64-bit sum and the single rounding of y leave, and
infinities and NaN in every operand."""
import numpy as np
import pytest

from snack_inputs import normal
from tests import ckpt_oracle as O
from tests.gpu_util import dev, host, lib, say

pytestmark = pytest.mark.gpu

EPS = 1e-6
TINY = 2.0 ** -149      # fp32's smallest step


def _rows(n, key):
    """Rows of ordinary size, of magnitudes spread over 2^120, whose squares pass fp32 at both ends, and of zeros."""
    x = normal((7, n), key)
    x[1] *= np.exp2((np.arange(n) * 37 % 121 - 60).astype(np.float32))
    x[2] *= np.float32(1e30)
    x[3] *= np.float32(1e36)
    x[4] *= np.float32(1e-30)
    x[5] = 0.0
    x[6, 0] = 1e25         # one value that hides the others
    return x


@pytest.mark.parametrize("n", [3, 40, 1023, 1030, 4999, 16400])
def test_y_and_rstd_are_rounded_once(n):
    """rstd is half a step of fp32 off.  y is half a step off, or where that is more the steps at which rstd's second
    part, the rest of h rstd and their products end (rstd below 2^-122 has no second part of its own)."""
    L = lib()
    x = _rows(n, f"normvalues/{n}")
    gain = (normal((n,), f"normvalues/{n}/g") * 3).astype(np.float32)
    say("rounded once", n)
    _, y, rstd, _ = L.rmsnorm_fwd(dev(x), dev(gain), EPS)
    yr, rr = O.norm_fwd(x, gain, np.float64(np.float32(EPS)))
    # 64 bits leave far less than a hundredth of a half step
    assert (np.abs(host(rstd) - rr) <= 1.01 * O.U32 * rr + TINY / 2).all()
    g = np.abs(gain.astype(np.float64))
    tol = 1.01 * O.U32 * np.abs(yr) + TINY * (1 + 3 * g) + TINY / 2 * np.abs(x.astype(np.float64)) * g
    bad = np.abs(host(y).astype(np.float64) - yr) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], host(y)[bad][:5], yr[bad][:5])


@pytest.mark.parametrize("n", [3, 77, 1030, 16400])
def test_forward_non_finite(n):
    """What an infinity or a NaN of h, of the residual or of the gain reaches, against the definition in 64 bits."""
    import torch
    L = lib()
    x, res = normal((6, n), f"normvalues/nf/{n}"), normal((6, n), f"normvalues/nf/{n}/r")
    gain = (1 + 0.1 * normal((n,), f"normvalues/nf/{n}/g")).astype(np.float32)
    x[0, 1], x[1, 2], res[2, 0], x[3, 0], res[3, 0] = np.inf, np.nan, -np.inf, np.inf, -np.inf
    say("forward clean gain", n)
    with np.errstate(invalid="ignore", over="ignore"):
        h = x + res
        for gn in (gain, np.where(np.arange(n) % 3 == 1, np.inf, np.where(np.arange(n) % 5 == 2, -np.inf, gain))):
            gn = gn.astype(np.float32)
            gn[-1] = np.nan
            H, y, rstd, ck = L.rmsnorm_fwd(dev(x), dev(gn), EPS, residual=dev(res), q_format=O.E4M3)
            assert np.array_equal(host(H), h, equal_nan=True)
            yr, rr = O.norm_fwd(h, gn, np.float64(np.float32(EPS)))
            got = host(y).astype(np.float64)
            assert np.array_equal(np.isnan(got), np.isnan(yr))
            inf = np.isinf(yr)
            assert np.array_equal(got[inf], yr[inf]) and np.isinf(yr[4:]).any() == np.isinf(gn).any()
            fin = np.isfinite(yr)
            assert (np.abs(got[fin] - yr[fin]) <= 1.01 * O.U32 * np.abs(yr[fin])).all()
            ok = np.isfinite(rr)
            assert np.array_equal(np.isnan(host(rstd)), ~ok)
            assert (np.abs(host(rstd)[ok] - rr[ok]) <= 1.01 * O.U32 * rr[ok]).all()
            q, s = O.pack(host(y), O.E4M3)
            assert np.array_equal(host(ck.s), s)
            assert torch.equal(ck.q.cpu() & 127, torch.from_numpy(q) & 127)


@pytest.mark.parametrize("kept", ["f32", "bf16", "int8"])
@pytest.mark.parametrize("rows,n", [(40, 77), (5000, 96), (1500, 1030), (6, 16400)])
def test_backward_non_finite(rows, n, kept):
    """A NaN or an infinity of h, dY or dR stays in its row of dX and its column of dgain; the rest keeps its bits."""
    import torch
    L = lib()
    key = f"normvalues/nfb/{rows}x{n}"
    x, dy, dr = (normal((rows, n), key + k) for k in ("/h", "/dy", "/dr"))
    gain = (1 + 0.1 * normal((n,), key + "/g")).astype(np.float32)
    rstd = (1 / np.sqrt((x.astype(np.float64) ** 2).mean(-1) + EPS)).astype(np.float32)

    def call(x, dy, dr):
        h = L.Ckpt.pack(dev(x), O.INT8) if kept == "int8" else dev(x, torch.bfloat16 if kept == "bf16" else None)
        return [host(t) for t in L.rmsnorm_bwd(h, dev(gain), dev(rstd), dev(dy), dR=dev(dr))]

    say("backward non finite", rows, n, kept)
    dx, dg = call(x, dy, dr)
    assert np.isfinite(dx).all() and np.isfinite(dg).all()
    x2, dy2, dr2 = x.copy(), dy.copy(), dr.copy()
    x2[1, 40], dy2[2, 3], dy2[3, 4], dr2[4, 5] = np.nan, np.nan, np.inf, -np.inf
    dx2, dg2 = call(x2, dy2, dr2)
    other = [i for i in range(rows) if i not in (1, 2, 3, 4)]
    assert np.array_equal(dx2[other], dx[other])
    assert not np.isfinite(dx2[1:4]).any()
    assert dx2[4, 5] == -np.inf and np.array_equal(np.delete(dx2[4], 5), np.delete(dx[4], 5))
    lost = {40, 3, 4} | (set(range(32, 64)) if kept == "int8" else set())      # a checkpoint loses x's block of 32
    keep = [c for c in range(n) if c not in lost]
    assert not np.isfinite(dg2[sorted(lost)]).any() and np.array_equal(dg2[keep], dg[keep])
