"""Measured cases of the attention half of a served or trained transformer block.

Between the query, key and value projections of a block and its output projection lie the norms and the rotary
positions of queries and keys, and the attention.  Served, the keys and values stay in a cache of 8 or 4 bits a value:
for every block of 32 consecutive features of one token's head one exponent byte s (the block's scale is 2^(s - 127))
and 32 codes, signed integers of at most 127 in magnitude (int8), e4m3 numbers of at most 448, or e2m1 numbers of at
most 6 (4 bits).  The scale is the smallest power of two that brings the block's largest |value| into that range.

  qk       norms of queries and keys for each head, with the position rotation in the same pass
  qk_bwd   its gradient
  put      the same pass on the way to a cache: q normed and rotated, k normed, rotated and kept, v kept
  attend   attention of a sequence's newest tokens, or of another sequence's, over such a cache

Cached keys and values are returned as the values they stand for, in bf16, which holds every such value exactly.
"""
import math

import torch

own = False

BLOCK = 32
EPS = 1e-6
BASE = 10000.0
TOP = {"int8": 127.0, "e4m3": 448.0, "e2m1": 6.0}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
TYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

# tokens: rows of the projections' output; seq: tokens of a sequence, whose positions start at `past`;
# hq, hk: heads of the queries, and of the keys and values; d: features of a head; rot: how many of them are rotated;
# factor: positions scaled for a context `factor` times as long as the one trained on

def listed():
    return [
        # one token on its way through a GPT-2-small block (12 heads of 64): latency
        {"name": "qk_token", "op": "qk", "tokens": 1, "seq": 1, "past": 700, "hq": 12, "hk": 12, "d": 64, "rot": 64,
         "layout": "half", "factor": 1, "norm": True, "x": "f32", "y": "f32"},
        # a long prompt with grouped heads, half of each head rotated, queries and keys handed on in bf16
        {"name": "qk_prompt", "op": "qk", "tokens": 8192, "seq": 8192, "past": 0, "hq": 32, "hk": 8, "d": 128, "rot": 64,
         "layout": "pairs", "factor": 4, "norm": True, "x": "f32", "y": "bf16"},
        # the backward pass of 1024 tokens of the GPT-2-small block
        {"name": "qk_bwd_block", "op": "qk_bwd", "tokens": 1024, "seq": 1024, "past": 0, "hq": 12, "hk": 12, "d": 64,
         "rot": 64, "layout": "half", "factor": 1, "norm": True, "x": "f32", "y": "f32"},
        # a ragged number of tokens, heads of 80 features of which 20 are rotated
        {"name": "qk_bwd_odd", "op": "qk_bwd", "tokens": 9001, "seq": 1333, "past": 0, "hq": 20, "hk": 4, "d": 80,
         "rot": 20, "layout": "half", "factor": 1, "norm": True, "x": "f32", "y": "f32"},
        # one token each of 64 sequences, kept in 4 bits
        {"name": "put_step", "op": "put", "tokens": 64, "seq": 1, "past": 2500, "hq": 32, "hk": 8, "d": 128, "rot": 128,
         "layout": "half", "factor": 4, "norm": True, "x": "f32", "y": "f32", "fmt": "e2m1", "page": 64},
        # prompts of the GPT-2-small block, kept in 8 bits
        {"name": "put_prompt", "op": "put", "tokens": 8192, "seq": 1024, "past": 0, "hq": 12, "hk": 12, "d": 64,
         "rot": 64, "layout": "half", "factor": 1, "norm": True, "x": "f32", "y": "f32", "fmt": "int8", "page": 128},
        # one token of one GPT-2-small stream: latency
        {"name": "attend_token", "op": "attend", "b": 1, "nq": 1, "len": 1000, "hq": 12, "hk": 12, "d": 64,
         "fmt": "int8", "page": 64, "causal": True, "x": "f32"},
        # a served batch of streams of different lengths, grouped heads, 4 bits
        {"name": "attend_batch", "op": "attend", "b": 64, "nq": 1, "len": 4096, "hq": 32, "hk": 8, "d": 128,
         "fmt": "e2m1", "page": 64, "causal": True, "x": "f32"},
        # one token over one very long context, 4 bits
        {"name": "attend_long", "op": "attend", "b": 1, "nq": 1, "len": 131072, "hq": 32, "hk": 8, "d": 128,
         "fmt": "e2m1", "page": 128, "causal": True, "x": "bf16"},
        # a few queries each over an encoder's states of other, ragged lengths
        {"name": "attend_cross", "op": "attend", "b": 7, "nq": 5, "len": 1999, "hq": 15, "hk": 3, "d": 80,
         "fmt": "e4m3", "page": 32, "causal": False, "x": "f32"},
        # a piece of a long prompt over what is cached of it
        {"name": "attend_chunk", "op": "attend", "b": 1, "nq": 512, "len": 8192, "hq": 32, "hk": 8, "d": 128,
         "fmt": "int8", "page": 64, "causal": True, "x": "bf16"},
        # whole prompts of the GPT-2-small block
        {"name": "attend_prompt", "op": "attend", "b": 4, "nq": 1024, "len": 1024, "hq": 12, "hk": 12, "d": 64,
         "fmt": "int8", "page": 128, "causal": True, "x": "f32"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk", "qk_bwd", "put", "attend", "attend"])
    d = rng.choice([32, 40, 48, 64, 64, 80, 96, 128, 128, 192, 256])
    hk = rng.choice([1, 2, 3, 4, 8, 12])
    hq = hk * rng.choice([1, 1, 2, 4, 5, 8])
    fmt = rng.choice(["int8", "e4m3", "e2m1"])
    page = rng.choice([32, 64, 128, 256])
    x = rng.choice(["f32", "f32", "bf16"])
    if op == "attend":
        while True:
            b, n = _log_int(rng, 1, 128), _log_int(rng, 1, 131072)
            nq = 1 if rng.random() < 0.6 else _log_int(rng, 1, min(n, 2048))
            if b * n * hk * d <= 64 * 4096 * 8 * 128 and b * nq * hq * n * d <= 512 * 32 * 8192 * 128:
                break
        return {"op": op, "b": b, "nq": nq, "len": n, "hq": hq, "hk": hk, "d": d, "fmt": fmt, "page": page,
                "causal": rng.random() < 0.8, "x": x}
    while True:
        tokens = _log_int(rng, 1, 16384)
        if tokens * (hq + hk) * d <= 8192 * 40 * 128:
            break
    seq = _log_int(rng, 1, tokens)
    case = {"op": op, "tokens": tokens, "seq": seq, "past": rng.choice([0, _log_int(rng, 1, 100000)]), "hq": hq, "hk": hk,
            "d": d, "rot": d if rng.random() < 0.6 else 2 * rng.randint(1, d // 2), "layout": rng.choice(["half", "pairs"]),
            "factor": rng.choice([1, 1, 4, 8]), "norm": rng.random() < 0.8, "x": x, "y": rng.choice(["f32", x])}
    if op == "put":
        case["fmt"], case["page"] = fmt, page
    return case


def _lens(case):
    """Tokens of each sequence in the cache: from about a twentieth of the largest length to all of it."""
    n, least = case["len"], case["nq"] if case["causal"] else 1
    return [max(least, n - (n * ((i * 7) % 16)) // 16) for i in range(case["b"])]


# ---------------------------------------------------------------------------
# the plain forms: the cache's format and the rotation in torch operations
# ---------------------------------------------------------------------------

def _encode(x, fmt):
    """x [..., d] fp32 -> (codes uint8 [..., 32 ceil(d/32)], two a byte for e2m1, exponent bytes [..., ceil(d/32)])."""
    b = torch.nn.functional.pad(x, (0, -x.shape[-1] % BLOCK)).unflatten(-1, (-1, BLOCK))
    mant, expo = torch.frexp(b.abs().amax(-1))          # amax = mant 2^expo, mant in [1/2, 1)
    low, edge = {"int8": (120, 127 / 128), "e4m3": (118, 448 / 512), "e2m1": (124, 6 / 8)}[fmt]
    s = (expo + low + (mant > edge).to(expo.dtype)).clamp(1, 254)
    v = torch.ldexp(b, (127 - s)[..., None])
    if fmt == "e2m1":
        a = v.abs()
        step = 0.5 + 0.5 * (a >= 2.0) + 1.0 * (a >= 4.0)
        a = (a / step).round() * step
        c = torch.where(a < 2.0, a * 2.0, torch.where(a < 4.0, a + 2.0, a * 0.5 + 4.0)).to(torch.uint8)
        c = (c + 8 * torch.signbit(v)).to(torch.uint8)
        q = c[..., 0::2] + 16 * c[..., 1::2]
    else:
        q = v.round().to(torch.int8) if fmt == "int8" else v.to(torch.float8_e4m3fn)
    return q.view(torch.uint8).flatten(-2), s.to(torch.uint8)


def _decode(q, s, fmt, d):
    """The values that codes and exponent bytes stand for, fp32 [..., d]."""
    if fmt == "e2m1":
        q = torch.stack([q & 15, q >> 4], -1).flatten(-2)
        v = torch.tensor(E2M1 + [-e for e in E2M1], device=q.device)[q.int()]
    else:
        v = q.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).float()
    return torch.ldexp(v.unflatten(-1, (-1, BLOCK)), (s.int() - 127)[..., None]).flatten(-2)[..., :d]


def _frequencies(case):
    """Radians a position turns each rotated pair by (64 bits), and what the rotation is multiplied with."""
    rot, factor = case["rot"], case["factor"]
    f = BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    if factor == 1:
        return f, 1.0
    # pairs of over 32 turns within the trained length are kept, those under one are stretched, the rest in between
    turns = _trained(case) * f / (2.0 * math.pi)
    w = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
    return f * (w + (1.0 - w) / factor), 0.1 * math.log(factor) + 1.0


def _trained(case):
    return max(1, (case["past"] + case["seq"]) // case["factor"])


def _rotate(y, cos, sin, layout, back=False):
    """The rotation by each token's angles, cos and sin [tokens, rot / 2], of y [tokens, heads, d]."""
    r = cos.shape[-1]
    c, s = cos[:, None], -sin[:, None] if back else sin[:, None]
    if layout == "half":
        a, b = y[..., :r], y[..., r:2 * r]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = y[..., 0:2 * r:2], y[..., 1:2 * r:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([turned, y[..., 2 * r:]], -1)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _values(shape, g, scale=1.0):
    """Normal values, one feature in 16 three times as large."""
    x = torch.randn(*shape, device="cuda", generator=g) * scale
    x[..., ::16] *= 3.0
    return x


def _paged(b, n, page, g):
    """Pages of b sequences of up to n tokens, in an order of their own: int32 [b, pages of a sequence]."""
    w = -(-n // page)
    return torch.randperm(b * w, device="cuda", generator=g).to(torch.int32).view(b, w)


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": case}
    hq, hk, d = case["hq"], case["hk"], case["d"]
    if case["op"] == "attend":
        b, page = case["b"], case["page"]
        st["table"] = _paged(b, case["len"], page, g)
        st["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
        st["k"] = _values((st["table"].numel() * page, hk, d), g)
        st["v"] = _values((st["table"].numel() * page, hk, d), g)
        st["q"] = _values((b * case["nq"], hq, d), g, 0.7).to(TYPE[case["x"]])
        return st
    # rows of the projections' output: queries, keys and values side by side
    t, seq = case["tokens"], case["seq"]
    x = _values((t, hq + 2 * hk, d), g, 1.5).to(TYPE[case["x"]])
    st["q"], st["k"], st["v"] = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    st["pos"] = (case["past"] + torch.arange(t, device="cuda") % seq).to(torch.int32)
    st["gq"] = 1.0 + 0.1 * torch.randn(d, device="cuda", generator=g) if case["norm"] else None
    st["gk"] = 1.0 + 0.1 * torch.randn(d, device="cuda", generator=g) if case["norm"] else None
    if case["op"] == "qk_bwd":
        st["dq"] = (torch.randn(t, hq, d, device="cuda", generator=g) / t).to(TYPE[case["y"]])
        st["dk"] = (torch.randn(t, hk, d, device="cuda", generator=g) / t).to(TYPE[case["y"]])
    if case["op"] == "put":       # the tokens' places in the cache; positions before `past` are other calls'
        page = case["page"]
        first = case["past"] % page
        table = _paged(-(-t // seq), first + seq, page, g).long()
        at = first + torch.arange(t, device="cuda") % seq
        st["pages"] = table.numel()
        st["slot"] = table[torch.arange(t, device="cuda") // seq, at // page] * page + at % page
    return st


def prepare(case, seed):
    """What a serving or training program keeps: inputs, the table of the rotation, the cache."""
    st = _inputs(case, seed)
    if own:
        import coo_spmm_amd as L
        fmt = {"int8": L.INT8, "e4m3": L.E4M3, "e2m1": L.E2M1}
        if case["op"] == "attend":
            st["cache"] = L.KVCache(st["table"].numel(), case["hk"], case["d"], fmt[case["fmt"]], page=case["page"])
            every = torch.arange(st["k"].shape[0], device="cuda")
            st["cache"].write(st.pop("k"), st.pop("v"), every)
            return st
        more = {} if case["factor"] == 1 else {"factor": float(case["factor"]), "trained": _trained(case),
                                               "amplitude": 0.1 * math.log(case["factor"]) + 1.0}
        st["rope"] = L.RopeTable.make(case["past"] + case["seq"], case["rot"], base=BASE,
                                      layout=L.ROPE_HALF if case["layout"] == "half" else L.ROPE_PAIRS, **more)
        if case["op"] == "put":
            st["cache"] = L.KVCache(st["pages"], case["hk"], case["d"], fmt[case["fmt"]], page=case["page"])
        return st
    if case["op"] == "attend":
        for name in ("k", "v"):
            st[name + "_code"], st[name + "_exp"] = _encode(st.pop(name), case["fmt"])
        return st
    f, amp = _frequencies(case)
    angle = torch.arange(case["past"] + case["seq"], device="cuda", dtype=torch.float64)[:, None] * f
    st["cos"], st["sin"] = (torch.cos(angle) * amp).float(), (torch.sin(angle) * amp).float()
    if case["op"] == "put":
        rows, per = st["pages"] * case["page"], -(-case["d"] // BLOCK)
        width = per * BLOCK // (2 if case["fmt"] == "e2m1" else 1)
        for name in ("k", "v"):
            st[name + "_code"] = torch.zeros(rows, case["hk"], width, dtype=torch.uint8, device="cuda")
            st[name + "_exp"] = torch.zeros(rows, case["hk"], per, dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _run_own(st):
    import coo_spmm_amd as L
    case = st["case"]
    if case["op"] == "qk":
        q, k = L.qk_rope_fwd(st["q"], st["k"], st["pos"], rope=st["rope"], q_gain=st["gq"], k_gain=st["gk"], eps=EPS,
                             dtype=TYPE[case["y"]])
        return {"q": q, "k": k}
    if case["op"] == "qk_bwd":
        dq, dk, dgq, dgk = L.qk_rope_bwd(st["q"], st["k"], st["pos"], st["dq"], st["dk"], rope=st["rope"],
                                         q_gain=st["gq"], k_gain=st["gk"], eps=EPS)
        return {"dq": dq, "dk": dk, "dgq": dgq, "dgk": dgk}
    if case["op"] == "put":
        q = st["cache"].write_rope(st["q"], st["k"], st["v"], st["pos"], st["slot"], rope=st["rope"], q_gain=st["gq"],
                                   k_gain=st["gk"], eps=EPS, dtype=TYPE[case["y"]])
        k, v = st["cache"].read(st["slot"], torch.bfloat16)
        return {"q": q, "kept_k": k, "kept_v": v}
    return {"out": st["cache"].attend(st["q"], st["table"], st["lens"], causal=case["causal"])}


def _normed(x, gain, dtype):
    x = x.to(dtype)
    if gain is None:
        return x
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * gain.to(dtype)


def _attend(st):
    case = st["case"]
    b, nq, hk, d = case["b"], case["nq"], case["hk"], case["d"]
    group = case["hq"] // hk
    table = st["table"].long()
    n = table.shape[1] * case["page"]
    slot = (table[..., None] * case["page"] + torch.arange(case["page"], device="cuda")).view(b, n)
    t = torch.arange(n, device="cuda")
    there = t < st["lens"][:, None]                                           # [b, n]
    k = _decode(st["k_code"][slot], st["k_exp"][slot], case["fmt"], d).permute(0, 2, 3, 1).contiguous()
    v = _decode(st["v_code"][slot], st["v_exp"][slot], case["fmt"], d).permute(0, 2, 1, 3)
    v = torch.where(there[:, None, :, None], v, 0.0).contiguous()
    q = st["q"].float().view(b, nq, hk, group, d).transpose(1, 2).reshape(b, hk, nq * group, d)
    s = (q @ k) / math.sqrt(d)
    seen = there[:, None]
    if case["causal"]:                                                        # query i sees the tokens up to its own
        seen = t <= (st["lens"][:, None] - nq + torch.arange(nq, device="cuda"))[..., None]
    seen = seen.expand(b, nq, n).repeat_interleave(group, 1)[:, None]
    s = torch.where(seen, s, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    out = (p @ v) / p.sum(-1, keepdim=True)
    return out.view(b, hk, nq, group, d).transpose(1, 2).reshape(b * nq, case["hq"], d).to(st["q"].dtype)


def run(st):
    if own:
        return _run_own(st)
    case = st["case"]
    if case["op"] == "attend":
        return {"out": _attend(st)}
    pos, layout, to = st["pos"].long(), case["layout"], TYPE[case["y"]]
    cos, sin = st["cos"][pos], st["sin"][pos]
    if case["op"] == "qk":
        return {"q": _rotate(_normed(st["q"], st["gq"], torch.float32), cos, sin, layout).to(to),
                "k": _rotate(_normed(st["k"], st["gk"], torch.float32), cos, sin, layout).to(to)}
    if case["op"] == "put":
        q = _rotate(_normed(st["q"], st["gq"], torch.float32), cos, sin, layout).to(to)
        # 64 bits: what is kept lies next to a border of its grid here and there
        k = _rotate(_normed(st["k"], st["gk"], torch.float64), cos.double(), sin.double(), layout).float()
        out = {"q": q}
        for name, y in (("k", k), ("v", st["v"].float())):
            st[name + "_code"][st["slot"]], st[name + "_exp"][st["slot"]] = _encode(y, case["fmt"])
            out["kept_" + name] = _decode(st[name + "_code"][st["slot"]], st[name + "_exp"][st["slot"]], case["fmt"],
                                          case["d"]).to(torch.bfloat16)
        return out
    out = {}
    for name in ("q", "k"):
        dy = _rotate(st["d" + name].float(), cos, sin, layout, back=True)
        x, gain = st[name].float(), st["g" + name]
        if gain is None:
            out["d" + name], out["dg" + name] = dy.to(st[name].dtype), None
            continue
        rstd = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
        xh, w = x * rstd, dy * gain
        out["d" + name] = (rstd * (w - xh * (w * xh).mean(-1, keepdim=True))).to(st[name].dtype)
        out["dg" + name] = (dy * xh).sum((0, 1))
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its exact results
# ---------------------------------------------------------------------------

def work(case):
    hq, hk, d = case["hq"], case["hk"], case["d"]
    size = {"f32": 4.0, "bf16": 2.0}
    if "fmt" in case:       # bytes of a token's key or value in the cache
        kept = hk * (d * (0.5 if case["fmt"] == "e2m1" else 1.0) + -(-d // BLOCK))
    if case["op"] == "attend":
        lens, nq = _lens(case), case["nq"]
        seen = sum(nq * n - (nq * (nq - 1) // 2 if case["causal"] else 0) for n in lens)
        return {"bytes": sum(lens) * 2.0 * kept + 2.0 * case["b"] * nq * hq * d * size[case["x"]]
                + 4.0 * (case["b"] + sum(-(-n // case["page"]) for n in lens)),
                "flops": 4.0 * seen * hq * d}
    t = case["tokens"]
    table = 4.0 * t + 4.0 * min(t, case["seq"]) * case["rot"] + (8.0 * d if case["norm"] else 0.0)
    e = float(t) * (hq + hk) * d
    if case["op"] == "qk":
        return {"bytes": e * (size[case["x"]] + size[case["y"]]) + table, "flops": 10.0 * e}
    if case["op"] == "qk_bwd":       # without the norms x is not read
        by = e * size[case["y"]] + e * size[case["x"]] * (2.0 if case["norm"] else 1.0)
        return {"bytes": by + table + (8.0 * d if case["norm"] else 0.0), "flops": 20.0 * e}
    x = float(t) * (hq + 2 * hk) * d         # q, k, v in, q out, the cache written, read back, its values in bf16
    return {"bytes": x * size[case["x"]] + float(t) * hq * d * size[case["y"]] + 4.0 * t * kept + 4.0 * t * hk * d
            + table + 8.0 * t, "flops": 10.0 * e + 6.0 * t * hk * d}


def _grid(x, fmt):
    """The nearest values of the blocks' grids, in 64 bits."""
    b = torch.nn.functional.pad(x.double(), (0, -x.shape[-1] % BLOCK)).unflatten(-1, (-1, BLOCK))
    most = b.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.ceil(torch.log2(most / TOP[fmt])).clamp_min(-126.0))
    v = b / scale
    if fmt == "int8":
        step = torch.ones_like(v)
    else:                   # fraction bits below the leading one, down to the smallest normal number
        bits, least = (3, -6) if fmt == "e4m3" else (1, 0)
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** least))) - bits)
    return (torch.round(v / step) * step * scale).flatten(-2)[..., :x.shape[-1]]


def _turn(y, angle, amp, layout, sign=1.0):
    """Each pair of y as a complex number times amp exp(i sign angle)."""
    r = angle.shape[-1]
    z = torch.polar(torch.full_like(angle, amp), sign * angle)[:, None]
    out = y.clone()
    first, second = (slice(0, r), slice(r, 2 * r)) if layout == "half" else (slice(0, 2 * r, 2), slice(1, 2 * r, 2))
    w = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * z
    out[..., first], out[..., second] = w.real, w.imag
    return out


def _exact_attend(case, st):
    nq, hk, d = case["nq"], case["hk"], case["d"]
    group = case["hq"] // hk
    outs = []
    for i, n in enumerate(_lens(case)):
        t = torch.arange(n, device="cuda")
        slot = st["table"][i].long()[t // case["page"]] * case["page"] + t % case["page"]
        k, v = _grid(st["k"][slot], case["fmt"]), _grid(st["v"][slot], case["fmt"])
        q = st["q"][i * nq:(i + 1) * nq].double()
        heads = []
        for h in range(case["hq"]):
            s = q[:, h] @ k[:, h // group].t().contiguous() * d ** -0.5
            if case["causal"]:
                s.masked_fill_(t[None] > (n - nq + torch.arange(nq, device="cuda"))[:, None], -math.inf)
            heads.append(torch.softmax(s, -1) @ v[:, h // group].contiguous())
        outs.append(torch.stack(heads, 1))
    return torch.cat(outs)


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "attend":
        return {"out": _exact_attend(case, st)}
    f, amp = _frequencies(case)
    angle, layout = st["pos"].double()[:, None] * f, case["layout"]

    def rms(x):
        return torch.sqrt(x.square().sum(-1, keepdim=True) / case["d"] + EPS)

    def turned(name):
        x, gain = st[name].double(), st["g" + name]
        return _turn(x if gain is None else gain.double() * x / rms(x), angle, amp, layout)

    if case["op"] == "qk":
        return {"q": turned("q"), "k": turned("k")}
    if case["op"] == "put":
        return {"q": turned("q"), "kept_k": _grid(turned("k"), case["fmt"]), "kept_v": _grid(st["v"].double(), case["fmt"])}
    out = {}
    for name in ("q", "k"):
        dy = _turn(st["d" + name].double(), angle, amp, layout, -1.0)
        x, gain = st[name].double(), st["g" + name]
        if gain is None:
            out["d" + name], out["dg" + name] = dy, None
            continue
        n = rms(x)
        w = dy * gain.double()
        out["d" + name] = w / n - x * (w * x).sum(-1, keepdim=True) / (case["d"] * n ** 3)
        out["dg" + name] = (dy * x / n).sum((0, 1))
    return out
