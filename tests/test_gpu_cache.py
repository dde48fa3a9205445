"""The cache of keys and values: what is written reads back as the format's nearest values, slots, and the pass that
norms and rotates on the way."""
import numpy as np
import pytest

from snack_inputs import normal
from tests import attend_oracle as A
from tests.gpu_util import dev, host, lib, say

pytestmark = pytest.mark.gpu

FMTS = [A.INT8, A.E4M3, A.E2M1]
DIMS = [1, 31, 32, 33, 64, 80, 96, 128, 130, 160, 192, 200, 256]


def _values(shape, key):
    x = normal(shape, key).astype(np.float32)
    x[..., ::9] *= 6.0
    x *= np.exp2((np.arange(shape[0]) * 11 % 61 - 30).astype(np.float32))[:, None, None]
    if shape[0] > 2:
        x[2] = 0.0
    return x


def _same(got, want, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    bad = ~((got == want) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} differ, first at {tuple(np.argwhere(bad)[0])}"


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", DIMS)
def test_write_and_read(d, fmt):
    """Every slot of a few pages in a shuffled order, some left out; the others keep what they held."""
    import torch
    L = lib()
    pages, page, heads = 3, 96, 3
    say("write", d, fmt)
    c = L.KVCache(pages, heads, d, fmt, page=page)
    n = pages * page
    rng = np.random.default_rng(d)
    first = rng.permutation(n)
    k0, v0 = _values((n, heads, d), f"cache/{d}/k0"), _values((n, heads, d), f"cache/{d}/v0")
    c.write(dev(k0), dev(v0), dev(first))
    some = rng.permutation(n)[:77]
    k1, v1 = _values((77, heads, d), f"cache/{d}/k1"), _values((77, heads, d), f"cache/{d}/v1")
    c.write(dev(k1), dev(v1), dev(some))
    want_k, want_v = np.zeros((n, heads, d)), np.zeros((n, heads, d))
    want_k[first], want_v[first] = A.grid(k0, fmt), A.grid(v0, fmt)
    want_k[some], want_v[some] = A.grid(k1, fmt), A.grid(v1, fmt)
    slot = dev(np.arange(n))
    k, v = c.read(slot)
    _same(host(k), want_k, "keys")
    _same(host(v), want_v, "values")
    kb, vb = c.read(slot, torch.bfloat16)
    _same(host(kb.float()), want_k, "keys in bf16")
    _same(host(vb.float()), want_v, "values in bf16")
    # bf16 input, as parts of wider rows
    x = torch.cat([dev(k0), dev(v0)], 1).to(torch.bfloat16)
    c.write(x[:, :heads], x[:, heads:], dev(first))
    k, v = c.read(dev(first))
    _same(host(k), A.grid(host(x[:, :heads].float()), fmt), "keys from bf16")
    _same(host(v), A.grid(host(x[:, heads:].float()), fmt), "values from bf16")


@pytest.mark.parametrize("fmt", FMTS)
def test_special_values_and_slots_outside(fmt):
    import torch
    L = lib()
    heads, d = 2, 70
    c = L.KVCache(2, heads, d, fmt, page=32)
    k = normal((6, heads, d), "cache/special").astype(np.float32)
    v = k[::-1].copy()
    k[0, 0, 5], k[1, 1, 69], v[2, 0, 33], v[3, 1, 0] = np.nan, np.inf, -np.inf, np.nan
    k[4], v[4] = -0.0, np.finfo(np.float32).tiny
    say("special", fmt)
    c.data.fill_(0x5A)
    before = c.data.clone()
    c.write(dev(k), dev(v), dev(np.array([-1, 64, 2 ** 40, -2 ** 62, 2 ** 31, 1 << 36])))
    torch.cuda.synchronize()
    assert torch.equal(c.data, before)            # nothing outside is written
    slots = np.array([63, 0, 31, 32, 5, 7])
    c.write(dev(k), dev(v), dev(slots))
    gk, gv = (host(t) for t in c.read(dev(slots)))
    _same(gk, A.grid(k, fmt), "keys")
    _same(gv, A.grid(v, fmt), "values")
    assert np.isnan(gk[0, 0, :32]).all() and np.isfinite(gk[0, 0, 32:]).all() and np.isnan(gk[1, 1, 64:]).all()
    gk, gv = (host(t) for t in c.read(dev(np.array([-1, 64, -2 ** 62, 2 ** 40]))))
    for g in (gk, gv):
        assert (g[[0, 2]] == 0).all() and np.isnan(g[[1, 3]]).all()
    e = c.read(dev(np.zeros(0, np.int64)))
    assert e[0].shape == (0, heads, d)
    c.write(dev(k[:0]), dev(v[:0]), dev(np.zeros(0, np.int64)))


@pytest.mark.parametrize("fmt", [A.INT8, A.E2M1])
def test_every_exponent(fmt):
    """Largest values on both sides of every border of the range, in every binade."""
    L = lib()
    top = 127.0 if fmt == A.INT8 else 6.0
    e = np.arange(-126, 120)
    x = np.zeros((len(e) * 3, 1, 32), np.float32)
    with np.errstate(under="ignore", over="ignore"):
        edge = np.float32(top) * np.exp2(e).astype(np.float32)
    x[0::3, 0, 3], x[1::3, 0, 3], x[2::3, 0, 3] = edge, np.nextafter(edge, np.float32(np.inf)), np.nextafter(edge, np.float32(0))
    x[:, 0, 4:9] = x[:, 0, 3:4] * np.array([0.999, 0.5, 0.126, -0.31, 0.011], np.float32)
    n = x.shape[0]
    say("exponents", fmt)
    c = L.KVCache(-(-n // 32), 1, 32, fmt, page=32)
    slot = dev(np.arange(n))
    c.write(dev(x), dev(x[::-1].copy()), slot)
    k, v = c.read(slot)
    _same(host(k), A.grid(x, fmt), "keys")
    _same(host(v), A.grid(x[::-1], fmt), "values")


def test_slots():
    """Against the definition, sequences of no token and pages that there are not among them."""
    L = lib()
    page, pages = 32, 9
    c = L.KVCache(pages, 1, 32, A.INT8, page=page)
    table = np.array([[3, 8, 0], [1, -1, 2], [4, 9, 5], [7, 6, 2 ** 31 - 1], [0, 0, 0]], np.int32)
    lens = np.array([70, 96, 40, 97, 0], np.int32)
    for starts in (np.array([0, 3, 3, 43, 60, 60], np.int32), np.array([2, 3, 100, 101, 198, 199], np.int32), None):
        t = 200 if starts is not None else 35
        say("slots", None if starts is None else starts.tolist())
        pos, slot = (host(x) for x in c.slots(dev(table), dev(lens), t, None if starts is None else dev(starts)))
        first = starts if starts is not None else np.arange(6) * 7
        want_p, want_s = np.zeros(t, np.int64), np.full(t, -1)
        for b in range(5):
            for i in range(first[b], first[b + 1]):
                p = lens[b] - first[b + 1] + i
                if p >= 0:
                    want_p[i] = p
                    if p // page < 3 and 0 <= table[b, p // page] < pages:
                        want_s[i] = table[b, p // page] * page + p % page
        assert np.array_equal(pos, want_p) and np.array_equal(slot, want_s)
    assert c.slots(dev(table), dev(lens), 0)[0].numel() == 0
    with pytest.raises(ValueError):
        c.slots(dev(table), dev(lens), 34)


@pytest.mark.parametrize("layout", [A.HALF, A.PAIRS])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("shape", [(1, 12, 12, 64, 64), (67, 8, 2, 128, 128), (130, 5, 5, 80, 20), (9, 6, 3, 200, 96),
                                   (40, 4, 1, 256, 256), (3, 2, 2, 30, 10)])
def test_write_rope(shape, fmt, layout):
    """q as qk_rope_fwd gives it, bit for bit; the cache holds what qk_rope_fwd's k and v are rounded to."""
    import torch
    L = lib()
    t, hq, hk, d, rot = shape
    key = f"cache/rope/{shape}"
    for xtype in (torch.float32, torch.bfloat16):
        x = dev(normal((t, hq + 2 * hk, d), key).astype(np.float32)).to(xtype)
        q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        rope = L.RopeTable(dev(A.table(300, rot).astype(np.float32)), layout)
        pos = dev((np.arange(t) * 13 % 300).astype(np.int32))
        gq, gk = (dev((1 + 0.1 * normal((d,), key + n)).astype(np.float32)) for n in "qk")
        c = L.KVCache(5, hk, d, fmt, page=32)
        slot = np.random.default_rng(t).permutation(160)[:t]
        if t > 2:
            slot[1] = -1
        say("write_rope", shape, fmt, layout, xtype)
        yq = c.write_rope(q, k, v, pos, dev(slot), rope, gq, gk, 1e-6, dtype=torch.float32)
        wq, wk = L.qk_rope_fwd(q, k, pos, rope, gq, gk, 1e-6, dtype=torch.float32)
        assert torch.equal(yq, wq)
        ck, cv = (host(z) for z in c.read(dev(slot)))
        live = slot >= 0
        _same(ck[live], A.grid(host(wk)[live], fmt), "keys")
        _same(cv[live], A.grid(host(v.float())[live], fmt), "values")
        # as two calls, and without norms and rotation of the keys
        c2 = L.KVCache(5, hk, d, fmt, page=32)
        c2.write(wk, v.float(), dev(slot))
        assert all(torch.equal(a, b) for a, b in zip(c.read(dev(slot)), c2.read(dev(slot))))
        c.write_rope(q, k, v, None, dev(slot), None, gq, None, 1e-6)
        _same(host(c.read(dev(slot))[0])[live], A.grid(host(k.float())[live], fmt), "keys as they came")


def test_pages_past_2_31_bytes():
    """The last page of a cache of over 4 GB."""
    import torch
    L = lib()
    heads, d, page = 8, 256, 256
    pages = (9 << 29) // (heads * page * 2 * (d + 8)) + 1
    say("large cache", pages)
    c = L.KVCache(pages, heads, d, A.INT8, page=page)
    assert c.nbytes > 9 << 29
    slot = np.array([0, pages * page - 1, pages * page - 256, (pages // 2) * page + 31])
    k, v = _values((4, heads, d), "cache/large/k"), _values((4, heads, d), "cache/large/v")
    c.write(dev(k), dev(v), dev(slot))
    gk, gv = c.read(dev(slot))
    _same(host(gk), A.grid(k, A.INT8), "keys")
    _same(host(gv), A.grid(v, A.INT8), "values")
    # attention over the last page alone
    q = dev(normal((1, 8, d), "cache/large/q").astype(np.float32))
    c.write(dev(np.repeat(k, 32, 0)), dev(np.repeat(v, 32, 0)), dev(pages * page - 256 + np.arange(128)))
    out = c.attend(q, dev(np.array([[pages - 1]], np.int32)), dev(np.array([128], np.int32)))
    kk, vv = A.grid(np.repeat(k, 32, 0), A.INT8), A.grid(np.repeat(v, 32, 0), A.INT8)
    want, mag, terms, top = A.attend(host(q), kk, vv, d ** -0.5, [127])
    assert (np.abs(host(out) - want) <= A.attend_tol(128, d, mag, terms, top) + 1e-37).all()
    del c
    torch.cuda.empty_cache()


def test_past_2_32_threads():
    """More heads than one launch takes (four lanes a head, 2^32 threads of keys and values): a few tokens written, all
    over the call, and all of them read."""
    import torch
    L = lib()
    t, h, d, page = (1 << 17) + 37, 4096, 2, 32
    assert 2 * 4 * t * h > 2 ** 32
    c = L.KVCache(4, h, d, A.E4M3, page=page)
    k, v = (torch.randn(t, h, d, device="cuda", dtype=torch.bfloat16) for _ in "kv")
    rows = torch.linspace(0, t - 1, 128, device="cuda").long()
    slot = torch.full((t,), -1, dtype=torch.int64, device="cuda")
    slot[rows] = torch.randperm(128, device="cuda")
    say("past 2^32 threads: write")
    c.write(k, v, slot)
    few = L.KVCache(4, h, d, A.E4M3, page=page)
    few.write(k[rows], v[rows], slot[rows])
    assert all(torch.equal(a, b) for a, b in zip(c.read(slot[rows]), few.read(slot[rows])))
    del k, v
    every = torch.arange(t, device="cuda") * 5 % 128
    say("past 2^32 threads: read")
    gk, gv = c.read(every, torch.bfloat16)
    wk, wv = c.read(every[:128], torch.bfloat16)
    n = t // 128 * 128
    assert all(torch.equal(g[:n].view(-1, 128, h, d), w.expand(n // 128, 128, h, d)) and torch.equal(g[n:], w[:t - n])
               for g, w in ((gk, wk), (gv, wv)))
    del gk, gv
    torch.cuda.empty_cache()
