"""Norms and rotation of queries and keys, the cache and the attention without a GPU: the oracle against closed forms
and differences, and every refusal that is decided on the host."""
import ctypes
import math
import os

import numpy as np
import pytest

from tests import attend_oracle as A


def _lib():
    import coo_spmm_amd as L
    if not os.path.exists(L.LIB_PATH):
        import __graft_entry__
        __graft_entry__._builder().build()
    return L


def test_oracle_e2m1_grid():
    """Largest value 6: no scale.  Halfway values go to the even code; a block with a NaN is NaN; scales are the
    smallest powers of two that hold the block."""
    x = np.zeros((5, 40), np.float32)
    x[0, :9] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0]
    x[1, :3] = [6.0001, 1.0, 3.0]
    x[2, 33] = np.nan
    x[3, :2] = [3.0, 0.3]
    x[4, 0] = 1e-45
    y = A.grid(x, A.E2M1)
    assert y[0, :9].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -4]
    assert y[1, :3].tolist() == [6, 1, 3]          # steps of 2^1: 3.00005 -> 3, 0.5 and 1.5 are numbers
    assert np.isnan(y[2, 32:]).all() and (y[2, :32] == 0).all()
    assert y[3, :2].tolist() == [3, 0.25]
    assert y[4, 0] == 0
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((50, 96)) * np.exp2(rng.integers(-30, 30, (50, 1)))).astype(np.float32)
    amax = np.abs(x.reshape(50, 3, 32)).max(-1)
    sc = np.exp2(np.ceil(np.log2(amax / 6.0)))
    step = np.repeat(sc, 32, 1) * np.where(np.abs(x) >= 4 * np.repeat(sc, 32, 1), 2, np.where(np.abs(x) >= 2 * np.repeat(sc, 32, 1), 1, 0.5))
    assert (np.abs(A.grid(x, A.E2M1) - x) <= step / 2).all()


def test_oracle_rotation():
    """A rotation keeps the pairs' lengths, its transpose undoes it, and the scores of rotated vectors depend on the
    distance of their positions alone."""
    rng = np.random.default_rng(2)
    tab = A.table(400, 12)
    x = rng.standard_normal((2, 1, 20))
    for layout in (A.HALF, A.PAIRS):
        y, _ = A.rotate(x, tab, np.array([17, 230]), layout)
        assert np.allclose((y * y).sum(-1), (x * x).sum(-1)) and np.allclose(A.rotate(y, tab, np.array([17, 230]), layout, True)[0], x)
        assert np.array_equal(y[..., 12:], x[..., 12:])
        q, k = x[:1], x[1:]
        dots = [(A.rotate(q, tab, np.array([p]), layout)[0] * A.rotate(k, tab, np.array([p + 9]), layout)[0]).sum() for p in (0, 3, 390)]
        assert np.allclose(dots, dots[0])
    # scaled by parts: fast pairs stay, slow ones are divided
    f = A.frequencies(64, 10000.0)
    g = A.frequencies(64, 10000.0, factor=4.0, trained=2048.0)
    turns = 2048.0 * f / (2 * math.pi)
    assert np.allclose(g[turns >= 32], f[turns >= 32]) and np.allclose(g[turns <= 1], f[turns <= 1] / 4)
    assert (np.diff(g) < 0).all() and np.allclose(A.frequencies(8, 100.0, factor=2.0), A.frequencies(8, 100.0) / 2)


def test_oracle_qk_gradient_against_differences():
    rng = np.random.default_rng(3)
    tab, pos = A.table(50, 6), np.array([3, 41])
    x, dy, g = rng.standard_normal((2, 3, 10)), rng.standard_normal((2, 3, 10)), 1 + 0.3 * rng.standard_normal(10)
    for layout in (A.HALF, A.PAIRS):
        for gain in (g, None):
            loss = lambda xx, gg: (A.qk_fwd(xx, gg, 1e-6, tab, pos, layout) * dy).sum()
            dx, dg, _, _ = A.qk_bwd(x, dy, gain, 1e-6, tab, pos, layout)
            for i in ((0, 0, 0), (1, 2, 4), (1, 0, 9)):
                e = np.zeros_like(x)
                e[i] = 1e-6
                assert abs((loss(x + e, gain) - loss(x - e, gain)) / 2e-6 - dx[i]) < 1e-7
            for i in (0, 7) if gain is not None else ():
                e = np.zeros_like(g)
                e[i] = 1e-6
                assert abs((loss(x, g + e) - loss(x, g - e)) / 2e-6 - dg[i]) < 1e-7


def test_oracle_attention_against_torch():
    import torch
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((3, 4, 6)), rng.standard_normal((9, 2, 6)), rng.standard_normal((9, 2, 6))
    out = A.attend(q, k, v, 0.4, [5, -1, 8])[0]
    assert (out[1] == 0).all()
    for i, n in ((0, 6), (2, 9)):
        for h in range(4):
            s = torch.from_numpy(k[:n, h // 2] @ q[i, h]) * 0.4
            assert np.allclose(torch.softmax(s, 0).numpy() @ v[:n, h // 2], out[i, h])


def _cache(L, **over):
    c = dict(data=4096, pages=4, page_tokens=64, heads=2, head_dim=64, fmt=L.INT8)
    c.update(over)
    return L._Cache(*(c[f] for f, _ in L._Cache._fields_))


def test_c_refusals():
    """Host-side checks: nothing is launched, so no device is needed (addresses are never followed)."""
    L = _lib()
    c, bad, uns, ws, ok = L._lib, L.ERR_INVALID_ARG, L.ERR_UNSUPPORTED, L.ERR_WORKSPACE, L.OK
    p, odd, one = 4096, 4098, 4097
    nan, inf = float("nan"), float("inf")
    ref = ctypes.byref
    tab = lambda n=8, rot=4, base=1e4, factor=1.0, trained=0.0, low=1.0, high=32.0, amp=1.0, t=p: \
        c.snack_rope_table(n, rot, base, factor, trained, low, high, amp, t, None)
    assert tab(n=0) == bad and tab(rot=3) == bad and tab(rot=0) == bad and tab(rot=258) == bad and tab(t=None) == bad
    assert tab(base=0.0) == bad and tab(base=inf) == bad and tab(factor=0.0) == bad and tab(factor=nan) == bad
    assert tab(trained=-1.0) == bad and tab(low=32.0) == bad and tab(high=inf) == bad and tab(amp=nan) == bad
    assert tab(t=odd) == bad and tab(n=2**31 - 1, rot=256) == uns

    good = L._Rope(p, 8, 4, L.ROPE_HALF)
    ropes = [L._Rope(None, 8, 4, 0), L._Rope(p, 0, 4, 0), L._Rope(p, 8, 3, 0), L._Rope(p, 8, 0, 0), L._Rope(p, 8, 66, 0),
             L._Rope(p, 8, 4, 2), L._Rope(odd, 8, 4, 0)]

    def fwd(Q=p, hq=2, K=p, hk=1, xf=L.F32, t=4, d=64, pos=p, rope=good, gq=p, gk=p, eps=1e-6, Yq=p, Yk=p, yf=L.F32):
        return c.snack_qk_rope_fwd(Q, hq * d, d, hq, K, hk * d, d, hk, xf, t, d, pos, None if rope is None else ref(rope),
                                   gq, gk, eps, Yq, Yk, yf, None)
    assert all(fwd(rope=r) == bad for r in ropes) and fwd(pos=None) == bad and fwd(pos=odd) == bad
    assert fwd(Q=None) == bad and fwd(K=None) == bad and fwd(Yq=None) == bad and fwd(Yk=None) == bad
    assert fwd(Q=odd) == bad and fwd(K=odd) == bad and fwd(Yq=odd) == bad and fwd(gq=odd) == bad and fwd(gk=odd) == bad
    assert fwd(Q=one, xf=L.BF16) == bad and fwd(Yk=one, yf=L.BF16) == bad
    assert fwd(xf=L.INT8) == bad and fwd(yf=L.E2M1) == bad and fwd(eps=-1.0) == bad and fwd(eps=nan) == bad and fwd(eps=inf) == bad
    assert fwd(d=0) == bad and fwd(d=257) == bad and fwd(t=-1) == bad and fwd(hq=-1) == bad and fwd(hq=0, hk=0) == bad
    assert fwd(t=1 << 31) == uns and fwd(t=1 << 28, hq=8) == uns and fwd(t=0, Q=None, Yq=None) == ok

    need = ctypes.c_int64()
    assert c.snack_qk_rope_bwd_work(4, 2, 1, 64, ctypes.byref(need)) == ok and need.value > 0
    assert c.snack_qk_rope_bwd_work(4, 2, 1, 64, None) == bad and c.snack_qk_rope_bwd_work(4, 2, 1, 300, ctypes.byref(need)) == bad

    def bwd(Q=p, hq=2, K=p, hk=1, xf=L.F32, t=4, d=64, pos=p, rope=good, gq=p, gk=p, eps=1e-6, dq=p, dk=p, yf=L.F32, dX=p,
            dXk=p, dgq=p, dgk=p, w=p, wb=1 << 24):
        return c.snack_qk_rope_bwd(Q, hq * d, d, hq, K, hk * d, d, hk, xf, t, d, pos, None if rope is None else ref(rope),
                                   gq, gk, eps, dq, hq * d, d, dk, hk * d, d, yf, dX, dXk, dgq, dgk, w, wb, None)
    assert all(bwd(rope=r) == bad for r in ropes) and bwd(pos=None) == bad
    assert bwd(Q=None) == bad and bwd(dq=None) == bad and bwd(dk=None) == bad and bwd(dX=None) == bad and bwd(dXk=None) == bad
    assert bwd(gq=None) == bad and bwd(gk=None) == bad        # a gradient is wanted of a gain that there is not
    assert bwd(w=None) == bad and bwd(w=odd) == bad and bwd(wb=16) == ws and bwd(xf=5) == bad and bwd(yf=L.INT8) == bad
    assert bwd(dq=odd) == bad and bwd(dX=odd) == bad and bwd(dgq=odd) == bad and bwd(eps=-1.0) == bad
    assert bwd(hq=0, hk=0) == bad and bwd(t=1 << 31) == uns

    size = lambda **o: (c.snack_cache_bytes(ref(_cache(L, **o)), ctypes.byref(need)), need.value)
    assert size() == (ok, 4 * 64 * 2 * 2 * (64 + 2)) and size(data=None)[0] == ok
    assert size(fmt=L.E2M1)[1] == 4 * 64 * 2 * 2 * (32 + 2) and size(fmt=L.E4M3)[1] == 4 * 64 * 2 * 2 * 66
    for over in (dict(pages=0), dict(page_tokens=0), dict(page_tokens=33), dict(page_tokens=16), dict(heads=0),
                 dict(head_dim=0), dict(head_dim=257), dict(fmt=L.F32), dict(fmt=5)):
        assert size(**over)[0] == bad, over
    assert size(pages=1 << 36)[0] == uns and size(heads=1 << 13)[0] == uns and size(page_tokens=1 << 30, heads=2, pages=1)[0] == uns
    assert c.snack_cache_bytes(None, ctypes.byref(need)) == bad and c.snack_cache_bytes(ref(_cache(L)), None) == bad

    def slots(cache=None, table=p, width=2, lens=p, starts=p, n=3, t=5, pos=p, slot=p):
        return c.snack_cache_slots(ref(cache or _cache(L)), table, width, lens, starts, n, t, pos, slot, None)
    assert slots(table=None) == bad and slots(width=0) == bad and slots(lens=None) == bad and slots(n=-1) == bad
    assert slots(starts=None) == bad and slots(starts=None, n=0) == bad and slots(pos=None) == bad and slots(slot=4100) == bad
    assert slots(t=-1) == bad and slots(t=0, pos=None, slot=None) == ok and slots(t=1 << 31) == uns

    def write(cache=None, K=p, V=p, xf=L.F32, t=4, slot=p):
        return c.snack_cache_write(ref(cache or _cache(L)), K, 128, 64, V, 128, 64, xf, t, slot, None)
    assert write(K=None) == bad and write(V=None) == bad and write(slot=None) == bad and write(slot=4100) == bad
    assert write(K=odd) == bad and write(V=odd) == bad and write(V=one, xf=L.BF16) == bad and write(xf=L.INT8) == bad
    assert write(cache=_cache(L, data=None)) == bad and write(cache=_cache(L, data=4104)) == bad and write(t=-1) == bad
    assert write(t=0, K=None, V=None, slot=None) == ok and write(t=1 << 30) == uns

    def wr(Q=p, hq=4, pos=p, slot=p, rope=good, Yq=p, yf=L.F32, eps=1e-6, t=4):
        return c.snack_cache_write_rope(ref(_cache(L)), Q, 256, 64, hq, p, 128, 64, p, 128, 64, L.F32, t, pos, slot,
                                        None if rope is None else ref(rope), p, p, eps, Yq, yf, None)
    assert all(wr(rope=r) == bad for r in ropes) and wr(Q=None) == bad and wr(Yq=None) == bad and wr(pos=None) == bad
    assert wr(slot=None) == bad and wr(yf=L.E4M3) == bad and wr(eps=nan) == bad and wr(eps=inf) == bad and wr(t=0, slot=None) == ok

    def read(cache=None, slot=p, t=4, K=p, V=p, yf=L.F32):
        return c.snack_cache_read(ref(cache or _cache(L)), slot, t, K, V, yf, None)
    assert read(slot=None) == bad and read(K=None, V=None) == bad and read(K=odd) == bad and read(V=one, yf=L.BF16) == bad
    assert read(yf=L.INT8) == bad and read(t=-1) == bad and read(t=0, slot=None) == ok and read(cache=_cache(L, data=None)) == bad

    work = lambda hq=4, t=4, n=2, cache=None: c.snack_cache_attend_work(ref(cache or _cache(L)), hq, t, n, ctypes.byref(need))
    assert work() == ok and need.value > 0 and work(hq=3) == bad and work(hq=0) == bad and work(t=-1) == bad and work(n=-1) == bad
    assert work(t=1 << 31) == uns and work(cache=_cache(L, fmt=0)) == bad

    def attend(cache=None, Q=p, hq=4, qf=L.F32, t=4, table=p, width=2, lens=p, starts=None, n=2, scale=0.1, out=p, w=p, wb=1 << 28):
        return c.snack_cache_attend(ref(cache or _cache(L)), Q, hq * 64, 64, hq, qf, t, table, width, lens, starts, n, scale,
                                    1, out, w, wb, None)
    assert attend(Q=None) == bad and attend(Q=odd) == bad and attend(hq=3) == bad and attend(hq=0) == bad and attend(qf=L.INT8) == bad
    assert attend(table=None) == bad and attend(width=0) == bad and attend(lens=None) == bad and attend(lens=odd) == bad
    assert attend(n=0) == bad and attend(n=3) == bad and attend(starts=odd) == bad and attend(n=-1) == bad
    assert attend(scale=0.0) == bad and attend(scale=-1.0) == bad and attend(scale=nan) == bad and attend(scale=inf) == bad
    assert attend(out=None) == bad and attend(out=odd) == bad and attend(w=None) == bad and attend(w=4104) == bad and attend(wb=64) == ws
    assert attend(cache=_cache(L, data=None)) == bad and attend(t=0, Q=None, out=None) == ok and attend(t=1 << 30) == uns
    assert attend(width=1 << 30) == uns and attend(starts=p, n=0) == ok


def test_python_refusals():
    import torch
    L = _lib()
    q, pos = torch.zeros(4, 2, 64), torch.zeros(4, dtype=torch.int32)
    for call in (lambda: L.qk_rope_fwd(q, None, q_gain=torch.ones(64)), lambda: L.qk_rope_bwd(q, None, pos, q, None),
                 lambda: L.RopeTable(torch.zeros(8, 4))):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        L.qk_rope_fwd(q.double(), None)
    with pytest.raises(TypeError):
        L.qk_rope_fwd(q.numpy(), None)
    for shape in ((4, 64), (4, 2, 300), (4, 0, 64)):
        with pytest.raises(ValueError):
            L.qk_rope_fwd(torch.zeros(shape), None)
    with pytest.raises(L.SnackError):
        L.KVCache(4, 2, 64, L.INT8, page=48)
    with pytest.raises(L.SnackError):
        L.KVCache(4, 2, 300, L.INT8)
    with pytest.raises(L.SnackError):
        L.KVCache.nbytes_of(4, 2, 64, L.BF16)
    with pytest.raises((ValueError, TypeError)):
        L.KVCache(4, 2, 64, L.INT8, data=torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(TypeError):
        L.KVCache(4, 2, 64, L.INT8, data=np.zeros(8))
    assert L.KVCache.nbytes_of(3, 2, 80, L.E2M1, page=32) == 3 * 2 * 32 * (2 * 48 + 3 + 4)


def test_cache_sizes_past_63_bits():
    """pages * page_tokens below 2^36, also where the product wraps to something small."""
    L = _lib()
    need = ctypes.c_int64()

    def size(pages, page, **o):
        return L._lib.snack_cache_bytes(ctypes.byref(_cache(L, pages=pages, page_tokens=page, heads=1, **o)), ctypes.byref(need))
    for pages, page in ((1 << 34, 1 << 30), (1 << 59, 32), ((1 << 63) - 1, 32), ((1 << 62) // 32 + 1, 1 << 7), (1 << 31, 32),
                        (1 << 6, 1 << 30)):
        assert size(pages, page) == L.ERR_UNSUPPORTED, (pages, page)
        with pytest.raises(L.SnackError):
            L.KVCache.nbytes_of(pages, 1, 64, L.INT8, page=page)
    for pages, page in (((1 << 31) - 1, 32), ((1 << 6) - 1, 1 << 30)):      # a token of 64 features: 2 (64 + 2) bytes
        assert size(pages, page) == L.OK and need.value == pages * page * 132


def test_largest_scale():
    """The exponents are taken to base 2: a scale whose product with log2(e) is no fp32 number is refused (a score of 0
    times it would be NaN); the largest other one gets as far as the workspace's check."""
    L = _lib()

    def attend(scale):
        p = 4096
        return L._lib.snack_cache_attend(ctypes.byref(_cache(L)), p, 128, 64, 2, L.F32, 2, p, 1, p, None, 2, scale, 1, p, p, 0, None)
    top = float(np.finfo(np.float32).max)
    assert attend(top) == L.ERR_INVALID_ARG and attend(top / math.log2(math.e) * (1 + 2.0 ** -20)) == L.ERR_INVALID_ARG
    assert attend(top / math.log2(math.e) * (1 - 2.0 ** -20)) == L.ERR_WORKSPACE
