"""Attention over the cache against 64 bits, one token to chunks, and what lies behind masks, lengths and pages."""
import numpy as np
import pytest

from snack_inputs import normal
from tests import attend_oracle as A
from tests.ckpt_oracle import U16, U32
from tests.gpu_util import dev, host, lib, say

pytestmark = pytest.mark.gpu

FMTS = [A.INT8, A.E4M3, A.E2M1]


class Case:
    """Sequences in shuffled pages (what no token was written to is garbage, codes of NaN among it), their keys and
    values, and a call's queries."""

    def __init__(self, lens, nqs, hq, hk, d, fmt, page, key, qtype="f32", spread=1.0, starts=True, pad=0):
        import torch
        L = lib()
        rng = np.random.default_rng(abs(hash((tuple(lens), hq, hk, d, fmt, page))) % (1 << 31))
        self.lens, self.nqs, self.hq, self.hk, self.d, self.fmt, self.page = lens, nqs, hq, hk, d, fmt, page
        n = len(lens)
        self.width = max(1, max(-(-x // page) for x in lens)) + 1
        used = [-(-x // page) for x in lens]
        pages = sum(used) + 2
        ids = rng.permutation(pages)
        self.table = np.full((n, self.width), -7, np.int32)       # behind the lengths: no pages
        at = 0
        for b in range(n):
            self.table[b, :used[b]] = ids[at:at + used[b]]
            at += used[b]
        self.cache = L.KVCache(pages, hk, d, fmt, page=page)
        self.cache.data.fill_(0xFF)                               # NaN codes and exponents
        self.k, self.v = [], []
        for b in range(n):
            k, v = normal((lens[b], hk, d), f"{key}/k{b}") * spread, normal((lens[b], hk, d), f"{key}/v{b}")
            k, v = k.astype(np.float32), v.astype(np.float32)
            self.write(b, k, v)
            self.k.append(A.grid(k, fmt))
            self.v.append(A.grid(v, fmt))
        self.t = sum(nqs) + pad
        self.qt = torch.float32 if qtype == "f32" else torch.bfloat16
        self.q = dev(normal((self.t, hq, d), f"{key}/q").astype(np.float32)).to(self.qt)
        self.starts = np.concatenate([[0], np.cumsum(nqs)]).astype(np.int32) if starts else None

    def slots(self, b, n):
        i = np.arange(n)
        return self.table[b][i // self.page].astype(np.int64) * self.page + i % self.page

    def write(self, b, k, v):
        if len(k):
            self.cache.write(dev(k), dev(v), dev(self.slots(b, len(k))))

    def run(self, causal=True, scale=None, **kw):
        return self.cache.attend(self.q, dev(self.table), dev(np.array(self.lens, np.int32)),
                                 None if self.starts is None else dev(self.starts), causal=causal, scale=scale, **kw)

    def check(self, out, causal=True, scale=None):
        scale = self.d ** -0.5 if scale is None else scale
        q, out = host(self.q.float()), host(out.float())
        at = 0
        for b, (n, nq) in enumerate(zip(self.lens, self.nqs)):
            limits = [n - nq + i if causal else n - 1 for i in range(nq)]
            want, mag, terms, top = A.attend(q[at:at + nq], self.k[b], self.v[b], scale, limits)
            got = out[at:at + nq]
            at += nq
            exact = self.q.dtype.itemsize == 4
            nb = -(-self.d // 32)
            tol = A.attend_tol(n, self.d, mag, terms, top, 0.0 if exact else 2.0 ** -17) + 1e-37
            if not exact:
                # more than 16 queries of a head: probabilities rounded to bf16
                tol = tol + 2 * U16 * mag + U16 * np.abs(want)
            bad = ~(np.abs(got - want) <= tol)
            assert not bad.any(), (f"sequence {b}: {int(bad.sum())} of {bad.size} off, first at {tuple(np.argwhere(bad)[0])}: "
                                   f"{got[tuple(np.argwhere(bad)[0])]} for {want[tuple(np.argwhere(bad)[0])]}")
            # independent roundings add up by their root: the whole sequence's error, relative, for fp32
            if exact and np.linalg.norm(want) > 0:
                most = 16 * U32 * (np.sqrt(96 * nb) * terms.max() + np.sqrt(n / 8 + 64))
                err = np.linalg.norm(got - want) / np.linalg.norm(want)
                assert err <= most, (b, err, most)


# lengths and new tokens of the sequences, query heads, cache heads, features, tokens of a page
CASES = [([1], [1], 1, 1, 1, 32), ([5], [1], 12, 12, 64, 64), ([32, 33, 31], [1, 1, 1], 8, 2, 128, 32),
         ([1000], [1], 12, 12, 64, 64), ([257, 3, 700], [1, 1, 1], 32, 2, 96, 96), ([64, 1], [4, 1], 15, 3, 80, 32),
         ([300, 40], [7, 40], 6, 3, 160, 64), ([97, 128, 5, 0], [17, 0, 5, 2], 4, 4, 200, 32), ([2100], [3], 16, 1, 256, 256),
         ([129] * 5, [1] * 5, 5, 1, 33, 128), ([70, 300], [2, 1], 2, 2, 192, 64), ([77, 20], [30, 3], 40, 2, 32, 32)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("i", range(len(CASES)))
def test_attend(i, fmt):
    lens, nqs, hq, hk, d, page = CASES[i]
    for qtype in ("f32", "bf16"):
        c = Case(lens, nqs, hq, hk, d, fmt, page, f"attend/{i}", qtype)
        for causal in (True, False):
            say("attend", CASES[i], fmt, qtype, causal)
            c.check(c.run(causal), causal)
    if len(set(nqs)) == 1:       # the same without starts
        import torch
        out = c.run()
        c.starts = None
        assert torch.equal(out, c.run())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,hq,hk", [(64, 12, 12), (128, 8, 2), (80, 4, 4)])
def test_chunks(d, hq, hk, fmt):
    """Many queries of a head: whole prompts, and a chunk over what was there before it."""
    for lens, nqs in (([200], [200]), ([150, 333, 64], [70, 129, 64]), ([90], [300])):
        for qtype in ("f32", "bf16"):
            c = Case(lens, nqs, hq, hk, d, fmt, 64, f"chunk/{d}", qtype)
            say("chunk", lens, nqs, d, fmt, qtype)
            c.check(c.run())
            c.check(c.run(False, 0.3), False, 0.3)


def test_long_context_is_split():
    """Runs of tiles over many workgroups, lengths at their edges."""
    for lens in ([4096 * 4 + 1], [20000, 1, 31, 5000, 64, 33], [2048] * 40):
        for fmt in (A.INT8, A.E2M1):
            c = Case(lens, [1] * len(lens), 4, 2, 64, fmt, 128, f"long/{len(lens)}")
            say("long", len(lens), fmt)
            c.check(c.run())


@pytest.mark.parametrize("nq", [1, 20, 132])
def test_more_units_than_workgroups(nq):
    """Short and long sequences of every kind of block, more of them than workgroups, some without a query."""
    rng = np.random.default_rng(nq)
    n = {1: 180, 20: 150, 132: 70}[nq]
    lens = [int(x) for x in rng.integers(1, 400, n)]
    lens[5], lens[6], lens[7] = 1900, 0, 2
    nqs = [nq] * n
    nqs[9], nqs[10] = 0, 0
    c = Case(lens, nqs, 4, 4, 32, A.E2M1, 32, f"units/{nq}")
    say("units", nq)
    c.check(c.run())


def test_large_scores():
    """Scores of hundreds: one token takes all the weight, maxima rise from tile to tile."""
    for spread, scale in ((30.0, None), (1.0, 25.0), (1e-3, None)):
        c = Case([700, 90], [1, 2], 4, 2, 64, A.E4M3, 64, f"large/{spread}", spread=spread)
        say("large scores", spread, scale)
        c.check(c.run(scale=scale), scale=scale)


def test_rising_maximum():
    """Keys whose score grows with their position, so that every tile raises the maximum, and falling ones."""
    for sign in (1.0, -1.0):
        c = Case([999], [1], 2, 1, 32, A.INT8, 32, "rising")
        c.q = dev(np.ones((1, 2, 32), np.float32))
        k = np.repeat(np.repeat(sign * np.arange(999, dtype=np.float32)[:, None, None] / 8, 32, 2), 1, 1)
        v = normal((999, 1, 32), "rising/v").astype(np.float32)
        c.write(0, k, v)
        c.k, c.v = [A.grid(k, A.INT8)], [A.grid(v, A.INT8)]
        say("rising", sign)
        c.check(c.run())


@pytest.mark.parametrize("nq", [1, 3, 40, 100])
@pytest.mark.parametrize("fmt", FMTS)
def test_what_is_not_seen_has_no_influence(fmt, nq):
    """NaN and infinities in keys and values that some queries see and others do not."""
    import torch
    n, hq, hk, d = 100, 4, 2, 64
    c = Case([n], [nq], hq, hk, d, fmt, 32, f"unseen/{nq}")
    clean = host(c.run())
    last = n - 1
    k, v = normal((1, hk, d), "unseen/k").astype(np.float32), normal((1, hk, d), "unseen/v").astype(np.float32)
    v[0, 1, 40] = np.nan                       # block 1 of head 1
    c.cache.write(dev(k), dev(v), dev(c.slots(0, n)[last:]))
    say("unseen value", fmt, nq)
    got = host(c.run())
    assert np.array_equal(got[:-1], clean[:-1])
    assert np.isnan(got[-1, 2:, 32:]).all() and np.isfinite(got[-1, :2]).all() and np.isfinite(got[-1, 2:, :32]).all()
    assert np.isnan(host(c.run(False))[:, 2:, 32:]).all()
    k[0, 0, 3] = np.inf
    v[0, 1, 40] = 0
    c.cache.write(dev(k), dev(v), dev(c.slots(0, n)[last:]))
    say("unseen key", fmt, nq)
    got = host(c.run())
    assert np.array_equal(got[:-1], clean[:-1]) and np.isnan(got[-1, :2]).all() and np.isfinite(got[-1, 2:]).all()
    if nq > 1:                                 # two tokens of the chunk, one seen by more queries
        v[0, 0, 0], k[0, 0, 3] = -np.inf, 0
        c.cache.write(dev(k), dev(v), dev(c.slots(0, n)[last - 1:last]))
        got = host(c.run())
        assert np.array_equal(got[:-2], clean[:-2]) and np.isnan(got[-2:, :2, :32]).all()


def test_rows_of_no_token_and_of_no_sequence():
    """Queries before the sequence's first token give 0, padding behind the last sequence keeps its bytes."""
    import torch
    c = Case([3, 0, 40], [5, 2, 1], 4, 2, 64, A.INT8, 32, "empty", pad=6)
    out = torch.full((c.t, 4, 64), 7.5, device="cuda")
    say("empty rows")
    r = c.run(out=out)
    assert r is out
    got = host(out)
    assert (got[:2] == 0).all() and (got[5:7] == 0).all() and (got[8:] == 7.5).all()
    c.check(out[:8])
    assert (host(c.run(False))[5:7] == 0).all()


def test_bad_pages_and_lengths():
    """A query that needs a page that there is not gets NaN, the others their results."""
    c = Case([100, 100, 64], [3, 1, 1], 4, 2, 64, A.E2M1, 32, "bad")
    clean = host(c.run())
    for page in (-1, 10 ** 6, 2 ** 31 - 1):
        t = c.table.copy()
        c.table = t.copy()
        c.table[1, 1] = page
        say("bad page", page)
        got = host(c.run())
        assert np.isnan(got[3]).all() and np.array_equal(got[:3], clean[:3]) and np.array_equal(got[4], clean[4])
        c.table = t
    lens = c.lens
    for n in (32 * c.width + 1, 10 ** 7, 2 ** 31 - 1):
        c.lens = [100, n, 64]
        say("length past the table", n)
        got = host(c.run())
        assert np.isnan(got[3]).all() and np.array_equal(got[:3], clean[:3]) and np.array_equal(got[4], clean[4])
    c.lens = [100, -5, 64]
    got = host(c.run())
    assert (got[3] == 0).all() and np.array_equal(got[:3], clean[:3])
    # the chunk's last page is bad: its first query does not see it
    c.lens = [97, 100, 64]
    keep = c.table[0, 3]
    want = host(c.run())
    c.table[0, 3] = -1
    got = host(c.run())
    c.table[0, 3] = keep
    assert np.isfinite(got[:2]).all() and np.array_equal(got[:2], want[:2]) and np.isnan(got[2]).all()
    c.lens = lens
    # starts that do not ascend, or leave the call's tokens: no access outside, and the tokens that one sequence alone
    # claims are right (token 2 is claimed by the first and the last)
    c.starts = np.array([-4, 3, 2, 1000], np.int32)
    say("bad starts")
    assert np.array_equal(host(c.run())[:2], clean[:2])


def test_shared_pages_and_strided_queries():
    import torch
    L = lib()
    c = Case([64, 70], [1, 1], 8, 4, 64, A.INT8, 32, "shared")
    c.table[1, :2] = c.table[0, :2]            # a common prefix
    c.k[1], c.v[1] = c.k[1].copy(), c.v[1].copy()
    c.k[1][:64], c.v[1][:64] = c.k[0], c.v[0]
    say("shared prefix")
    out = c.run()
    c.check(out)
    wide = torch.zeros(2, 11, 80, device="cuda")
    q = wide[:, 2:10, 5:69]
    q.copy_(c.q)
    c.q = q
    assert torch.equal(out, c.run())
    b = torch.zeros(2, 11, 80, device="cuda", dtype=torch.bfloat16)
    b[:, 2:10, 5:69] = q
    one = c.cache.attend(b[:, 2:10, 5:69], dev(c.table), dev(np.array(c.lens, np.int32)), dev(c.starts))
    two = c.cache.attend(b[:, 2:10, 5:69].contiguous(), dev(c.table), dev(np.array(c.lens, np.int32)), dev(c.starts))
    assert torch.equal(one, two)


def test_repeats_streams_and_two_calls_at_once():
    import torch
    cs = [Case([3000, 200], [1, 1], 8, 2, 128, A.E2M1, 64, f"twice/{i}") for i in range(2)]
    want = [c.run() for c in cs]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in cs]
    say("two streams")
    for _ in range(5):
        got = [c.run(stream=s) for c, s in zip(cs, ss)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_captured_step_follows_the_sequences():
    """A serving step (slots, norms, rotation, cache, attention) in a graph: replays take the lengths, pages and inputs of
    their time; a second graph and eager calls in between do not disturb it."""
    import torch
    L = lib()
    n, hq, hk, d, page, width = 5, 8, 2, 64, 32, 6
    c = L.KVCache(n * width, hk, d, L.E2M1, page=page)
    table = dev(np.random.default_rng(0).permutation(n * width).astype(np.int32).reshape(n, width))
    lens = dev(np.array([1, 30, 64, 100, 31], np.int32))
    every = dev(np.arange(n * width * page))
    c.write(dev(normal((n * width * page, hk, d), "step/k").astype(np.float32)), dev(normal((n * width * page, hk, d), "step/v").astype(np.float32)), every)
    x = dev(normal((n, hq + 2 * hk, d), "step/x").astype(np.float32))
    rope = L.RopeTable.make(width * page, d)
    gq, gk = torch.rand(d, device="cuda") + 0.5, torch.rand(d, device="cuda") + 0.5

    def step():
        pos, slot = c.slots(table, lens, n)
        q = c.write_rope(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], pos, slot, rope, gq, gk)
        return c.attend(q, table, lens)
    step()
    torch.cuda.synchronize()
    say("capture step")
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    for i in range(6):
        lens.add_(1)
        x.mul_(1.01).add_(0.01)
        if i == 3:
            table.copy_(table.flip(0))
        held = c.data.clone()
        graphs[i % 2].replay()
        got = outs[i % 2].clone()
        torch.cuda.synchronize()
        after = c.data.clone()
        c.data.copy_(held)
        want = step()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(after, c.data), i


@pytest.mark.parametrize("fmt", FMTS)
def test_served_tokens_equal_the_whole_sequence(fmt):
    """The operators together, as they are used: a prompt in one chunk, then tokens one at a time, against 64 bits over
    the whole sequence; the tokens one at a time also against the prompt's pass over all of them."""
    import torch
    L = lib()
    n, prompt, hq, hk, d, rot, page = 60, 41, 6, 2, 64, 32, 32
    key = "serve"
    x = [normal((n, hq + 2 * hk, d), f"{key}/{b}").astype(np.float32) for b in range(2)]
    gq, gk = ((1 + 0.1 * normal((d,), key + s)).astype(np.float32) for s in "qk")
    rope = L.RopeTable.make(n, rot, layout=L.ROPE_PAIRS, factor=4.0, trained=16.0)
    tab = host(rope.table)
    cache, whole = (L.KVCache(6, hk, d, fmt, page=page) for _ in range(2))
    table = dev(np.array([[4, 1], [0, 5]], np.int32))

    def run(c, rows, lens, starts=None):
        xt = dev(np.concatenate(rows))
        lt = dev(np.array(lens, np.int32))
        pos, slot = c.slots(table, lt, xt.shape[0], starts)
        q = c.write_rope(xt[:, :hq], xt[:, hq:hq + hk], xt[:, hq + hk:], pos, slot, rope, dev(gq), dev(gk))
        return host(c.attend(q, table, lt, starts))
    say("serve", fmt)
    got = [[], []]
    out = run(cache, [x[0][:prompt], x[1][:7]], [prompt, 7], dev(np.array([0, prompt, prompt + 7], np.int32)))
    got[0].append(out[:prompt])
    got[1].append(out[prompt:])
    for i in range(n - prompt):
        out = run(cache, [x[0][prompt + i:prompt + i + 1], x[1][7 + i:8 + i]], [prompt + i + 1, 8 + i])
        got[0].append(out[:1])
        got[1].append(out[1:])
    m = [n, 7 + n - prompt]
    full = run(whole, [x[0], x[1][:m[1]]], m, dev(np.array([0, m[0], m[0] + m[1]], np.int32)))
    for b in range(2):
        pos = np.arange(m[b])
        q64 = A.qk_fwd(x[b][:m[b], :hq], gq, np.float64(np.float32(1e-6)), tab, pos, A.PAIRS).astype(np.float32)
        k64 = A.qk_fwd(x[b][:m[b], hq:hq + hk], gk, np.float64(np.float32(1e-6)), tab, pos, A.PAIRS).astype(np.float32)
        want, mag, terms, top = A.attend(q64, A.grid(k64, fmt), A.grid(x[b][:m[b], hq + hk:], fmt), d ** -0.5, pos)
        # as in Case.check; q64 rounds like the kernel's q up to a step, which adds a step of every term
        tol = np.expm1(2 * ((6 * 32 * 2 * U32 * 2 + 8 * U32) * terms + 20 * U32) + 150 * 2 * U32)[..., None] * mag
        one = np.concatenate(got[b])
        assert (np.abs(one - want) <= tol).all() and (np.abs(full[m[0] * b:m[0] * b + m[b]] - want) <= tol).all()


@pytest.mark.parametrize("nq", [1, 5, 24, 70])
@pytest.mark.parametrize("fmt", FMTS)
def test_bf16_queries_lose_no_more_than_the_output_does(fmt, nq):
    """Blocks of 16, 64 and 256 queries of a cache head (4, 20, 96 and 280 of them here): a probability is the sum of two
    bf16 numbers in each.  The first is cut off, so the rest is below 2^(e - 7) of a probability from 2^e on, and its own
    rounding, half a step of 8 bits, below 2^(e - 16).  Beside that and fp32's sums only the output is rounded."""
    for d, causal in ((64, True), (128, False)):
        c = Case([600], [nq], 8, 2, d, fmt, 64, f"bf16/{nq}", "bf16")
        say("bf16 queries", fmt, nq, d)
        got, q = host(c.run(causal).float()), host(c.q.float())
        limits = [600 - nq + i if causal else 599 for i in range(nq)]
        want, mag, terms, top = A.attend(q, c.k[0], c.v[0], d ** -0.5, limits)
        tol = A.attend_tol(600, d, mag, terms, top, 2.0 ** -16)
        tol = U16 * (np.abs(want) + tol) + tol + 2.0 ** -133
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), f"{int(bad.sum())} of {bad.size} off, at most by {np.max(np.abs(got - want) / tol)} of the tolerance"


# tokens, query heads, cache heads, sequences: blocks of 64, 16 and 256 queries; more blocks than 32 bits hold
@pytest.mark.parametrize("tokens,hq,hk,n", [(200, 32, 8, 14), (1024, 1, 1, 64), (1024, 4, 1, 9), (1 << 16, 8, 1, (1 << 17) + 1)])
def test_starts_that_claim_tokens_many_times(tokens, hq, hk, n):
    """Starts 0, T, 0, T, ... claim all tokens over and over: more units than the workspace has entries for.  Nothing
    behind it is written, nor any result; the same call with starts that ascend, in the same workspace, is right."""
    import torch
    L = lib()
    d, page = 32, 32
    c = L.KVCache(2, hk, d, A.INT8, page=page)
    k, v = (normal((64, hk, d), "claims/" + s).astype(np.float32) for s in "kv")
    c.write(dev(k), dev(v), dev(np.arange(64)))
    q = dev(normal((min(tokens, 1024), hq, d), "claims/q").astype(np.float32)).repeat(-(-tokens // 1024), 1, 1)
    assert q.shape[0] == tokens
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda").repeat(n, 1)
    lens = torch.full((n,), 50, dtype=torch.int32, device="cuda")
    starts = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    starts[1::2] = tokens
    nbytes, guard = L.snack_cache_attend_work(c._ref, hq, tokens, n), 1 << 20
    room = torch.full((nbytes + guard,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((tokens, hq, d), 7.5, device="cuda")

    def run(s):
        L.snack_cache_attend(c._ref, q, L.F32, table, lens, s, d ** -0.5, False, out, room[:nbytes])
        torch.cuda.synchronize()
        assert (room[nbytes:] == 0xA5).all()
    say("claims", tokens, hq, hk, n)
    run(starts)
    assert (out == 7.5).all()
    starts[:] = tokens
    starts[0] = 0
    run(starts)
    rows = np.concatenate([np.arange(32) + 32, np.arange(18)])
    want, mag, terms, top = A.attend(host(q[:3]), A.grid(k, A.INT8)[rows], A.grid(v, A.INT8)[rows], d ** -0.5, [49] * 3)
    assert (np.abs(host(out[:3]) - want) <= A.attend_tol(50, d, mag, terms, top) + 1e-37).all()
    step = min(tokens, 1024)
    assert all(torch.equal(out[i:i + step], out[:step]) for i in range(step, tokens, step))


@pytest.mark.parametrize("nq", [3, 8, 40, 140])
@pytest.mark.parametrize("fmt", FMTS)
def test_a_large_score_of_another_query_has_no_influence(fmt, nq):
    """The newest token's key gives its own query, which alone sees it, a score far above all others: the queries before
    it, in the same block, keep every bit."""
    import torch
    n, hq, hk, d = 200, 4, 2, 64
    for qtype in ("f32", "bf16"):
        c = Case([n], [nq], hq, hk, d, fmt, 32, f"another/{nq}", qtype)
        outs = []
        for size in (0.0, 20.0):
            k = host(c.q.float())[-1:, ::hq // hk] * size
            c.cache.write(dev(k), dev(np.ones((1, hk, d), np.float32)), dev(c.slots(0, n)[-1:]))
            say("another", fmt, nq, qtype, size)
            outs.append(c.run())
        assert torch.equal(outs[0][:-1], outs[1][:-1])
        assert not torch.equal(outs[0][-1], outs[1][-1])


# query heads of a cache head, most new tokens of a sequence: blocks of 16, 64 and 256 queries (on average 2, 26, 160 of them)
@pytest.mark.parametrize("group,most", [(1, 3), (4, 15), (32, 11)])
def test_runs_of_sequences_and_of_blocks(group, most):
    """More sequences, and more blocks of queries, than a workgroup has threads (512 at most): ragged, runs of them
    without a query in the middle and at the end; then equally many queries of each, with and without starts."""
    import torch
    rng = np.random.default_rng(group)
    n = 700
    lens, nqs = rng.integers(1, 70, n), rng.integers(1, most + 1, n)
    lens[rng.permutation(n)[:20]] = 0
    nqs[100:180], nqs[-40:] = 0, 0
    mean = int(nqs.sum()) * group / n
    assert mean <= 16 if group == 1 else 16 < mean <= 128 if group == 4 else mean > 128
    assert (nqs > 0).sum() > 512
    c = Case(lens.tolist(), nqs.tolist(), group, 1, 32, A.INT8, 32, f"runs/{group}")
    say("runs", group)
    c.check(c.run())
    nq = max(1, most // 2 + 1)
    c.q = c.q[:nq * n] if c.q.shape[0] >= nq * n else torch.cat([c.q, c.q])[:nq * n].contiguous()
    c.nqs, c.starts = [nq] * n, (np.arange(n + 1) * nq).astype(np.int32)
    say("runs of equal sequences", group)
    out = c.run()
    c.check(out)
    c.starts = None
    assert torch.equal(out, c.run())


def test_sequences_without_a_query_cost_little():
    """A padded batch: 4000 sequences without a query behind eight with one, against the same in front of them, which
    gives the same bits.  (Walked one by one they took twenty times as long.)"""
    import torch
    live, n = 8, 4008
    c = Case([300] * live, [1] * live, 4, 2, 64, A.INT8, 32, "padded")
    table = np.full((n, c.width), -1, np.int32)
    times, outs = [], []
    for front in (True, False):
        at = n - live if front else 0
        t, lens = table.copy(), np.zeros(n, np.int32)
        t[at:at + live], lens[at:at + live] = c.table, 300
        args = (c.q, dev(t), dev(lens), dev(np.clip(np.arange(n + 1) - at, 0, live).astype(np.int32)))
        say("padded", front)
        outs.append(c.cache.attend(*args))
        spans = []
        for _ in range(20):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(5):
                c.cache.attend(*args)
            b.record()
            torch.cuda.synchronize()
            spans.append(a.elapsed_time(b))
        times.append(sorted(spans)[len(spans) // 2])
    c.check(outs[0])
    assert torch.equal(*outs) and times[1] < 4 * times[0], times


@pytest.mark.parametrize("n", [40, 3000])
@pytest.mark.parametrize("nq", [1, 20, 140])
def test_scores_that_are_all_minus_infinity(nq, n):
    """They have no softmax: NaN, and not the 0 of a query that sees nothing; the other queries keep every bit.  Results
    of one workgroup, and joined from many."""
    import torch
    for qtype in ("f32", "bf16"):
        c = Case([n], [nq], 2, 1, 32, A.INT8, 32, f"minus/{nq}/{n}", qtype)
        c.write(0, np.abs(normal((n, 1, 32), "minus/k")).astype(np.float32) + np.float32(0.5), normal((n, 1, 32), "minus/v").astype(np.float32))
        clean = [c.run(False), c.run()]
        assert all(x.isfinite().all() for x in clean)
        for value, at in ((-np.inf, 3), (-3e38, slice(None)), (np.inf, 3), (np.nan, 3)):
            q = c.q.clone()
            c.q[-1, 1, at] = value
            say("minus infinity", nq, n, qtype, value)
            for causal in (False, True):
                got = c.run(causal)
                assert got[-1, 1].isnan().all()
                got[-1, 1], want = 0, clean[causal].clone()
                want[-1, 1] = 0
                assert torch.equal(got, want)
            c.q = q
        # half of the queries before the sequence's first token: they see nothing.  (Over 40 tokens the length of 70 passes
        # what was written: those that see past it get NaN.)
        c.lens = [nq // 2]
        got = host(c.run().float())
        sees = np.arange(nq) - (nq - nq // 2)
        assert (got[sees < 0] == 0).all() and np.isfinite(got[sees < n]).all() and np.isnan(got[sees >= n]).all()
