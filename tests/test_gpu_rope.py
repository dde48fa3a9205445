"""Norms and rotation of queries and keys, and their gradient, against 64 bits.  Tolerances are sums of the roundings
(u = 2^-24, half a step of fp32, relative; 2^-8 of bf16) along the longest chain."""
import numpy as np
import pytest

from snack_inputs import normal
from tests import attend_oracle as A
from tests.ckpt_oracle import U16, U32
from tests.gpu_util import dev, host, lib, say

pytestmark = pytest.mark.gpu

# tokens, query heads, key heads, features, rotated: one of each; odd widths; pairs that share a lane's eight features;
# every group of lanes (up to 32, 64, 128, 256 features) and its edges; more heads than one workgroup takes
SHAPES = [(1, 1, 1, 1, 0), (1, 12, 12, 64, 64), (3, 2, 1, 2, 2), (5, 3, 1, 7, 4), (2, 4, 2, 31, 30), (7, 5, 5, 33, 6),
          (4, 8, 2, 80, 20), (70, 6, 2, 96, 48), (9, 4, 4, 128, 128), (3, 2, 2, 129, 22), (6, 3, 1, 256, 256),
          (400, 20, 4, 40, 36), (33, 2, 1, 200, 64)]


def _close(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first at {i}: {got[i]} for {want[i]}, "
                             f"tolerance {np.broadcast_to(tol, bad.shape)[i]}")


def _case(shape, key, xtype="f32"):
    """q, k as parts of one projection's rows; a table of 64 positions and the tokens' positions; gains."""
    import torch
    t, hq, hk, d, rot = shape
    x = normal((t, hq + 2 * hk, d), key + "/x")
    x *= np.exp2((np.arange(t) * 5 % 41 - 20).astype(np.float32))[:, None, None]      # rows of every magnitude
    if t > 2:
        x[2] = 0.0
    xt = dev(x.astype(np.float32), torch.bfloat16 if xtype == "bf16" else torch.float32)
    q, k = xt[:, :hq], xt[:, hq:hq + hk]
    tab = A.table(64, max(rot, 2)).astype(np.float32)
    pos = ((np.arange(t) * 7) % 64).astype(np.int32)
    gq, gk = (1 + 0.1 * normal((d,), key + "/g" + n).astype(np.float32) for n in "qk")
    return q, k, tab, pos, gq.astype(np.float32), gk.astype(np.float32)


def _out_tol(y, ytype):
    # fp32: one rounding of a value computed in 64 bits (and what is below the normal numbers); bf16: that and its own
    return U32 * np.abs(y) * (1 + 2.0 ** -20) + 2.0 ** -149 if ytype == "f32" else (U16 + 2 * U32) * np.abs(y) + 2.0 ** -133


@pytest.mark.parametrize("layout", [A.HALF, A.PAIRS])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, layout):
    import torch
    L = lib()
    t, hq, hk, d, rot = shape
    eps = np.float32(1e-6)
    for xtype, ytype in (("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")):
        q, k, tab, pos, gq, gk = _case(shape, f"rope/{shape}", xtype)
        rope = L.RopeTable(dev(tab), layout) if rot else None
        say("qk fwd", shape, layout, xtype, ytype)
        yq, yk = L.qk_rope_fwd(q, k, dev(pos), rope, dev(gq), dev(gk), float(eps), dtype=torch.float32 if ytype == "f32" else torch.bfloat16)
        for got, x, g in ((yq, q, gq), (yk, k, gk)):
            want = A.qk_fwd(host(x.float()), g, np.float64(eps), tab if rot else None, pos, layout)
            assert got.is_contiguous()
            # the rotation's sum of two products may cancel: 64 bits' error of its terms, some 10 roundings of 2^-53
            _close(host(got.float()), want, _out_tol(want, ytype) + 2.0 ** -48 * np.abs(want).max(-1, keepdims=True), "y")
    # rotation alone, norm of one of them alone, queries alone
    q, k, tab, pos, gq, gk = _case(shape, f"rope/{shape}")
    if rot:
        rope = L.RopeTable(dev(tab), layout)
        yq, yk = L.qk_rope_fwd(q, k, dev(pos), rope)
        for got, x in ((yq, q), (yk, k)):
            y64 = host(x).astype(np.float64)
            want, mag = A.rotate(y64, tab, pos, layout)
            _close(host(got), want, U32 * np.abs(want) * (1 + 2.0 ** -20) + 2.0 ** -51 * mag + 2.0 ** -149, "rotated")
        one, none = L.qk_rope_fwd(q, None, dev(pos), rope)
        assert none is None and torch.equal(one, yq)
    yq, yk = L.qk_rope_fwd(q, k, q_gain=dev(gq), eps=float(eps))
    assert torch.equal(yk, k) and not torch.equal(yq, q) or t * d == 0 or d == 1


def _bwd_case(shape, layout, xtype, ytype, gains, key):
    import torch
    L = lib()
    t, hq, hk, d, rot = shape
    q, k, tab, pos, gq, gk = _case(shape, key, xtype)
    dt = torch.float32 if ytype == "f32" else torch.bfloat16
    dq, dk = (dev(normal((t, h, d), key + n).astype(np.float32), dt) for h, n in ((hq, "/dq"), (hk, "/dk")))
    rope = L.RopeTable(dev(tab), layout) if rot else None
    say("qk bwd", shape, layout, xtype, ytype, gains)
    g = (dev(gq), dev(gk)) if gains else (None, None)
    return (q, k, tab, pos, gq, gk, dq, dk), L.qk_rope_bwd(q, k, dev(pos), dq, dk, rope, *g, 1e-6)


@pytest.mark.parametrize("layout", [A.HALF, A.PAIRS])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, layout):
    L = lib()
    t, hq, hk, d, rot = shape
    for xtype, ytype, gains in (("f32", "f32", True), ("f32", "bf16", True), ("bf16", "bf16", True), ("bf16", "f32", False)):
        if not gains and not rot:
            continue
        (q, k, tab, pos, gq, gk, dq, dk), got = _bwd_case(shape, layout, xtype, ytype, gains, f"ropeb/{shape}")
        for x, dy, g, gx, gg, h in ((q, dq, gq, got[0], got[2], hq), (k, dk, gk, got[1], got[3], hk)):
            dx, dg, ax, ag = A.qk_bwd(host(x.float()), host(dy.float()), g if gains else None, np.float64(np.float32(1e-6)),
                                      tab if rot else None, pos, layout)
            assert gx.dtype == x.dtype and gx.is_contiguous()
            # dy: product and fused sum; w; rstd, m, the fused difference, the last product; bf16's own where written
            tol = 9 * U32 * ax + 2.0 ** -140
            _close(host(gx.float()), dx, tol if xtype == "f32" else tol + U16 * np.abs(dx) + 2.0 ** -133, "dx")
            if not gains:
                assert gg is None
                continue
            # a lane's heads one after the other (a workgroup of 256 threads takes 4 to 64 heads at once, and at least
            # a sixth of 1280 workgroups share them out), its workgroup's 64, then 64 bits; 6 of each term
            chain = -(-t * h // (4 * 200)) + 64 + 6
            _close(host(gg), dg, chain * U32 * ag, "dgain")
    if rot:     # queries alone give the same
        (q, k, tab, pos, gq, gk, dq, dk), got = _bwd_case(shape, layout, "f32", "f32", True, f"ropeb/{shape}")
        alone = L.qk_rope_bwd(q, None, dev(pos), dq, None, L.RopeTable(dev(tab), layout), dev(gq), None, 1e-6)
        assert alone[1] is None and alone[3] is None and np.array_equal(host(alone[0]), host(got[0]))


@pytest.mark.parametrize("layout", [A.HALF, A.PAIRS])
def test_backward_against_differences(layout):
    """The gradient of a sum of the forward pass's own outputs, by differences of the forward pass in fp32."""
    import torch
    L = lib()
    t, hq, hk, d, rot = 3, 2, 1, 24, 12
    rng = np.random.default_rng(8)
    q, k = (dev(rng.standard_normal((t, h, d)).astype(np.float32)) for h in (hq, hk))
    wq, wk = (dev(rng.standard_normal((t, h, d)).astype(np.float32)) for h in (hq, hk))
    gq, gk = (dev((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)) for _ in "qk")
    pos = dev(np.array([3, 60, 11], np.int32))
    rope = L.RopeTable(dev(A.table(64, rot).astype(np.float32)), layout)

    def loss():
        yq, yk = L.qk_rope_fwd(q, k, pos, rope, gq, gk, 1e-6)
        return float((yq.double() * wq).sum() + (yk.double() * wk).sum())
    got = L.qk_rope_bwd(q, k, pos, wq, wk, rope, gq, gk, 1e-6)
    say("differences", layout)
    for x, grad in zip((q, k, gq, gk), got):
        for i in range(0, x.numel(), 7):
            v, e = float(x.view(-1)[i]), 2.0 ** -7
            x.view(-1)[i] = v + e
            a = loss()
            x.view(-1)[i] = v - e
            b = loss()
            x.view(-1)[i] = v
            # outputs of size ~3 rounded to 2^-23: 150 of them, over 2^-6; the third derivative times e^2 / 6
            assert abs((a - b) / (2 * e) - float(grad.view(-1)[i])) < 150 * 3 * U32 * 64 * 0.5 + 40 * e * e / 6, i


def test_table():
    """Every way to scale it, against 64 bits: one rounding, and angles up to 2^17 radians that hold 64 bits' 2^-53 of
    them times a few (the power, the product)."""
    L = lib()
    for n, rot, kw in ((1, 2, {}), (1000, 64, {}), (131072, 6, {}), (300, 128, dict(base=5e5)),
                       (500, 64, dict(factor=4.0, amplitude=1.25)), (900, 32, dict(factor=8.0, trained=128.0)),
                       (900, 96, dict(factor=2.0, trained=400.0, low=2.0, high=7.0, amplitude=0.5))):
        say("table", n, rot, kw)
        rope = L.RopeTable.make(n, rot, **kw)
        want = A.table(n, rot, **{"base": 10000.0, **kw})
        amp = kw.get("amplitude", 1.0)
        _close(host(rope.table), want, U32 * np.abs(want) + amp * n * 2.0 ** -47 + 2.0 ** -60, "table")
        assert (rope.positions, rope.rot) == (n, rot)


def test_positions_outside_the_table_and_special_values():
    import torch
    L = lib()
    t, h, d = 6, 2, 64
    x = normal((t, h, d), "rope/special").astype(np.float32)
    x[1, 0, 3], x[2, 1, 40], x[3, 0, 0] = np.inf, np.nan, 1e30
    pos = np.array([5, 5, 5, 5, 64, -1], np.int32)
    tab = A.table(64, 32).astype(np.float32)
    ones = torch.ones(d, device="cuda")
    for layout in (A.HALF, A.PAIRS):
        say("special", layout)
        rope = L.RopeTable(dev(tab), layout)
        y = host(L.qk_rope_fwd(dev(x), None, dev(pos), rope, ones)[0])
        assert np.isnan(y[4:]).all()                         # outside the table: the whole row
        assert np.isfinite(y[0]).all() and np.isfinite(y[1, 1]).all() and np.isfinite(y[2, 0]).all()
        assert np.isnan(y[2, 1]).all()                       # a NaN is in the mean
        assert np.isfinite(y[3]).all() and abs(y[3, 0, 0]) > 1
        # an infinity makes its head's other features 0, itself NaN, and its pair with it
        at = [3, 19] if layout == A.HALF else [2, 3]
        assert np.isnan(y[1, 0, at]).all() and (np.delete(y[1, 0], at) == 0).all()
        # rotation alone: only the pair of a special value has it
        y = host(L.qk_rope_fwd(dev(x), None, dev(pos), rope)[0])
        assert np.isfinite(np.delete(y[1, 0], at)).all() and not np.isfinite(y[1, 0, at]).any()
        assert np.isnan(y[2, 1, 40]) and np.isfinite(np.delete(y[2, 1], 40)).all()
        assert np.isnan(y[4:]).all()
        g = L.qk_rope_bwd(dev(x), None, dev(pos), dev(x), None, rope, None)
        assert np.isnan(host(g[0])[4:]).all() and np.isfinite(host(g[0])[0]).all()


def test_strides_streams_and_repeats():
    """Heads that lie apart, a broadcast head, another stream; the same bits every time; nothing written past the end."""
    import torch
    L = lib()
    t, hq, hk, d = 37, 6, 2, 80
    big = dev(normal((t, 3 * hq, 2 * d + 5), "rope/stride").astype(np.float32))
    q, k = big[:, 1::3, 3:3 + d], big[:, 2:3, 7:7 + d].expand(t, hk, d)
    gq, gk = torch.rand(d, device="cuda") + 0.5, torch.rand(d, device="cuda") + 0.5
    pos = dev((np.arange(t) % 50).astype(np.int32))
    rope = L.RopeTable(dev(A.table(50, 40).astype(np.float32)), A.HALF)
    torch.cuda.synchronize()
    say("strides")
    want = L.qk_rope_fwd(q.contiguous(), k.contiguous(), pos, rope, gq, gk)
    got = L.qk_rope_fwd(q, k, pos, rope, gq, gk)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    dq, dk = big[:, ::3, 1:1 + d], big[:, :hk, 2:2 + d]
    want = L.qk_rope_bwd(q.contiguous(), k.contiguous(), pos, dq.contiguous(), dk.contiguous(), rope, gq, gk)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (None, s, s):
        got = L.qk_rope_bwd(q, k, pos, dq, dk, rope, gq, gk, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    # nothing to do
    e = L.qk_rope_fwd(q[:0], k[:0], pos[:0], rope, gq, gk)
    assert e[0].shape == (0, hq, d) and e[1].shape == (0, hk, d)
    z = L.qk_rope_bwd(q[:0], k[:0], pos[:0], dq[:0], dk[:0], rope, gq, gk)
    assert (z[2] == 0).all() and (z[3] == 0).all()


def test_captured_gradient_beside_an_eager_one():
    import torch
    L = lib()
    t, hq, hk, d = 700, 8, 2, 64
    q, k, dq, dk = (dev(normal((t, h, d), f"rope/graph{i}").astype(np.float32)) for i, h in enumerate((hq, hk, hq, hk)))
    gq, gk = torch.rand(d, device="cuda") + 0.5, torch.rand(d, device="cuda") + 0.5
    pos = dev((np.arange(t) % 50).astype(np.int32))
    rope = L.RopeTable(dev(A.table(50, 64).astype(np.float32)), A.HALF)
    out = [torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(gq), torch.zeros_like(gk)]
    L.qk_rope_bwd(q, k, pos, dq, dk, rope, gq, gk)
    torch.cuda.synchronize()
    say("capture qk bwd")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for o, r in zip(out, L.qk_rope_bwd(q, k, pos, dq, dk, rope, gq, gk)):
            o.copy_(r)
    for i in range(3):
        q.mul_(1.1)
        pos.add_(1).remainder_(50)
        gk.mul_(0.9)
        for o in out:
            o.zero_()
        g.replay()
        eager = L.qk_rope_bwd(q, k, pos, dq, dk, rope, gq, gk)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager)), i


def test_past_2_31_values():
    """Offsets past 32 bits: a thousand copies of the same tokens give a thousand times the same rows."""
    import torch
    L = lib()
    t, h, d, n = 70, 128, 256, 1000
    base = dev(normal((t, h, d), "rope/large").astype(np.float32)).to(torch.bfloat16)
    x = base.repeat(n, 1, 1)
    assert x.numel() > 2 ** 31
    pos = (torch.arange(t * n, device="cuda") % t).to(torch.int32)
    rope = L.RopeTable.make(t, 64)
    gain = torch.rand(d, device="cuda") + 0.5
    say("past 2^31")
    y = L.qk_rope_fwd(x, None, pos, rope, gain)[0].view(n, t, h, d)
    want = L.qk_rope_fwd(base, None, pos[:t], rope, gain)[0]
    assert all(torch.equal(y[i], want) for i in (0, n // 2, n - 2, n - 1))
    del y
    dx, _, dg, _ = L.qk_rope_bwd(x, None, pos, x, None, rope, gain)
    wx, _, wg, _ = L.qk_rope_bwd(base, None, pos[:t], base, None, rope, gain)
    dx = dx.view(n, t, h, d)
    assert all(torch.equal(dx[i], wx) for i in (0, n // 2, n - 2, n - 1))
    # sums of n times as many terms, each side within its own chain of roundings of the terms' magnitudes (above): heads
    # of a lane (4 to a workgroup of 256 at 64 lanes, 8 at 32; 1280 workgroups), its workgroup's, 6 of each term
    dq = host(base.float())
    ag = A.qk_bwd(dq, dq, host(gain), 1e-6, A.table(t, 64), np.arange(t), A.HALF)[3]
    chain = -(-t * n * h // (4 * 1280)) + 64 + 6
    _close(host(dg), n * host(wg).astype(np.float64), 2 * n * chain * U32 * ag, "dgain")
    del x, dx
    torch.cuda.empty_cache()


def test_past_2_32_threads():
    """More heads than one launch takes (four lanes a head, 2^32 threads), against the same call in parts."""
    import torch
    L = lib()
    t, h, d = (1 << 17) + 37, 8192, 2
    assert 4 * t * h > 2 ** 32 and t * h < 2 ** 31
    q = dev(normal((1, h, d), "rope/threads").astype(np.float32)).to(torch.bfloat16).expand(t, h, d)
    k = dev(normal((t, 1, d), "rope/threads/k").astype(np.float32)).to(torch.bfloat16)
    rope = L.RopeTable.make(1000, 2)
    pos = (torch.arange(t, device="cuda") * 7 % 1000).to(torch.int32)
    gain = torch.tensor([0.5, 1.5], device="cuda")
    say("past 2^32 threads")
    yq, yk = L.qk_rope_fwd(q, k, pos, rope, gain, gain)
    step = 20011
    for i in range(0, t, step):
        wq, wk = L.qk_rope_fwd(q[i:i + step], k[i:i + step], pos[i:i + step], rope, gain, gain)
        assert torch.equal(yq[i:i + step], wq) and torch.equal(yk[i:i + step], wk), i
    del yq, wq
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rot", [0, 16])
def test_backward_of_rows_whose_rms_leaves_fp32(rot):
    """Without eps, rows down to the smallest numbers (1 / rms passes 2^128), up to the largest, between ordinary ones;
    a gradient past fp32 is the infinity of its sign.  An infinity makes its head's dx NaN and its feature's dgain alone."""
    import torch
    L = lib()
    t, h, d = 40, 2, 24
    rng = np.random.default_rng(rot)
    e = np.array([-149, -148, -140, -133, -129, -128, -127, -126, -125, -100, -1, 0, 60, 100, 126, 127])[np.arange(t) % 16]
    x = np.clip(rng.standard_normal((t, h, d)), -1.9, 1.9) * np.exp2(e.astype(np.float64))[:, None, None]
    x = x.astype(np.float32)
    x[..., 0] = np.exp2(e.astype(np.float64)).astype(np.float32)[:, None]      # no row of zeros
    g = (1 + 0.1 * rng.standard_normal(d)).astype(np.float32)
    tab, pos = A.table(64, 16).astype(np.float32) if rot else None, np.arange(t) % 64
    rope = L.RopeTable(dev(tab), A.HALF) if rot else None

    def bwd(x, dy):
        return [host(a) for a in L.qk_rope_bwd(dev(x), None, dev(pos.astype(np.int32)), dev(dy), None, rope, dev(g), eps=0.0)[::2]]
    for size in (1.0, 2.0 ** -30, 2.0 ** -70):
        dy = (rng.standard_normal((t, h, d)) * size).astype(np.float32)
        say("rms", rot, size)
        gx, gg = bwd(x, dy)
        dx, dg, ax, ag = A.qk_bwd(x, dy, g, 0.0, tab, pos, A.HALF)
        # as test_backward's; rstd of the largest rows is below the normal numbers, 2^-127: off by 2^-22 of itself
        tol = 13 * U32 * ax + 2.0 ** -140
        top = np.float64(np.finfo(np.float32).max)
        past, near = np.abs(dx) > top + 2 * tol, np.abs(dx) > top - 2 * tol
        assert (gx[past] == np.copysign(np.inf, dx[past])).all()
        _close(gx[~near], dx[~near], tol[~near], "dx")
        _close(gg, dg, (10 + 64 + 10) * U32 * ag, "dgain")
    x[3, 1, 5] = np.inf
    gx, gg = bwd(x, dy)
    assert np.isnan(gx[3, 1]).all() and np.isfinite(gx[3, 0]).all() and np.isnan(gg[5]) and np.isfinite(np.delete(gg, 5)).all()
