"""Measured cases of the residual RMS norm and of the 8-bit activation checkpoints.

A sparse layer's weights are a few per cent of a dense one's, so what a training step keeps in memory is its
activations.  The operators here keep them in 8 bits: a checkpoint of X [rows, n] holds, for every block of 32
consecutive features of a row, one exponent byte s (the block's scale is 2^(s - 127)) and one byte per value (a signed
integer, or an e4m3 number).  The scale is the smallest power of two that brings the block's largest |value| to at most
127 (integers) or 448 (e4m3).

  norm_fwd   h = x + residual, y = h / rms(h) * gain, and y's checkpoint
  norm_bwd   its gradient, h held in fp32, bf16 or as a checkpoint
  pack       a checkpoint made and read back
  gelu_fwd   exact GELU that leaves the checkpoints of its input and of its output
  gelu_bwd   its gradient from the input's checkpoint
  layer_bwd  a sparse layer's gradients (dW at the stored positions; dX) with its input read from a checkpoint

Checkpoints are returned as the values they stand for, in bf16, which holds every such value exactly.
"""
import math

import torch

own = False

BLOCK = 32
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token on its way through a GPT-2-small block: latency
        {"name": "norm_fwd_token", "op": "norm_fwd", "rows": 1, "n": 768, "h": "f32", "fmt": "int8"},
        # a long batch of wide hidden states with a bf16 residual stream
        {"name": "norm_fwd_wide", "op": "norm_fwd", "rows": 8192, "n": 5000, "h": "bf16", "fmt": "e4m3"},
        # 1024 tokens of the GPT-2-small block, the norm's input kept in 8 bits
        {"name": "norm_bwd_block", "op": "norm_bwd", "rows": 1024, "n": 768, "h": "int8", "fmt": "int8"},
        # ragged rows of odd width, fp32 residual stream
        {"name": "norm_bwd_odd", "op": "norm_bwd", "rows": 3333, "n": 4999, "h": "f32", "fmt": "int8"},
        # the input of a 500-wide layer at batch 64
        {"name": "pack_small", "op": "pack", "rows": 64, "n": 500, "fmt": "e4m3"},
        # a long batch of the 10000-wide layer's input
        {"name": "pack_large", "op": "pack", "rows": 4096, "n": 10000, "fmt": "int8"},
        # the GELU between the two layers of the GPT-2-small block, 1024 tokens
        {"name": "gelu_fwd_block", "op": "gelu_fwd", "rows": 1024, "n": 3072, "fmt": "int8"},
        # its backward on a long batch of a wider layer
        {"name": "gelu_bwd_wide", "op": "gelu_bwd", "rows": 6000, "n": 5000, "fmt": "e4m3"},
        # the smallest layer, one row: latency
        {"name": "layer_bwd_row", "op": "layer_bwd", "M": 500, "K": 500, "sparsity": 95, "rows": 1, "dx": True,
         "fmt": "int8"},
        # the GPT-2-small block's first layer, 1024 tokens
        {"name": "layer_bwd_up", "op": "layer_bwd", "M": 3072, "K": 768, "sparsity": 90, "rows": 1024, "dx": True,
         "fmt": "int8"},
        # its second layer at high sparsity, a ragged number of tokens
        {"name": "layer_bwd_down", "op": "layer_bwd", "M": 768, "K": 3072, "sparsity": 99, "rows": 1000, "dx": True,
         "fmt": "e4m3"},
        # the 10000 x 10000 layer as a first layer (no input gradient), batch 64
        {"name": "layer_bwd_large", "op": "layer_bwd", "M": 10000, "K": 10000, "sparsity": 95, "rows": 64,
         "dx": False, "fmt": "int8"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "pack", "gelu_fwd", "gelu_bwd", "layer_bwd"])
    fmt = rng.choice(["int8", "e4m3"])
    if op == "layer_bwd":
        while True:
            M, K, rows = _log_int(rng, 200, 10000), _log_int(rng, 200, 10000), _log_int(rng, 1, 2048)
            if M * K * max(rows, 64) <= 10000 * 10000 * 64:
                break
        return {"op": op, "M": M, "K": K, "sparsity": rng.choice([90, 93, 95, 98, 99]), "rows": rows,
                "dx": rng.random() < 0.5, "fmt": fmt}
    while True:
        rows, n = _log_int(rng, 1, 16384), _log_int(rng, 33, 10000)
        if rows * n <= 4096 * 10000 and n != 3072:
            break
    case = {"op": op, "rows": rows, "n": n, "fmt": fmt}
    if op == "norm_fwd":
        case["h"] = rng.choice(["f32", "bf16"])
    if op == "norm_bwd":
        case["h"] = rng.choice(["f32", "bf16", "int8", "e4m3"])
    return case


# ---------------------------------------------------------------------------
# the checkpoint's definition in torch operations
# ---------------------------------------------------------------------------

def _blocks(x):
    rows, n = x.shape
    return torch.nn.functional.pad(x, (0, -n % BLOCK)).reshape(rows, -1, BLOCK)


def _encode(x, fmt):
    """x [rows, n] fp32 -> (bytes [rows, 32 ceil(n/32)], exponent bytes [rows, ceil(n/32)])."""
    b = _blocks(x)
    mant, expo = torch.frexp(b.abs().amax(-1))          # amax = mant 2^expo, mant in [1/2, 1)
    if fmt == "int8":
        s = expo + 120 + (mant > 127 / 128).to(expo.dtype)
    else:
        s = expo + 118 + (mant > 448 / 512).to(expo.dtype)
    s = s.clamp(1, 254)
    v = torch.ldexp(b, (127 - s)[..., None])
    q = v.round().to(torch.int8) if fmt == "int8" else v.to(torch.float8_e4m3fn)
    return q.view(torch.uint8).reshape(x.shape[0], -1), s.to(torch.uint8)


def _decode(q, s, fmt, n):
    """The values a checkpoint stands for, fp32 [rows, n]."""
    v = q.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).float().reshape(*s.shape, BLOCK)
    return torch.ldexp(v, (s.int() - 127)[..., None]).reshape(q.shape[0], -1)[:, :n]


def _kept(x, fmt):
    """x after a round trip through a checkpoint, in bf16 (exact)."""
    return _decode(*_encode(x, fmt), fmt, x.shape[1]).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _hidden(rows, n, g, scale=1.0):
    """Hidden states: normal, with one feature in 64 four times as large."""
    x = torch.randn(rows, n, device="cuda", generator=g) * scale
    x[:, ::64] *= 4.0
    return x


def _support(case, g):
    """Distinct stored positions drawn uniformly, in row-major order, and their values."""
    M, K = case["M"], case["K"]
    nnz = M * K * (100 - case["sparsity"]) // 100
    pos = torch.randint(M * K, (nnz + nnz // 5 + 64,), device="cuda", generator=g).unique()
    pos = pos[torch.randperm(pos.numel(), device="cuda", generator=g)[:nnz]].sort().values
    vals = torch.randn(nnz, device="cuda", generator=g) / math.sqrt(nnz / M)
    return (pos // K).to(torch.int32), (pos % K).to(torch.int32), vals


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, rows, fmt = case["op"], case["rows"], case["fmt"]
    st = {"case": case}
    if op == "layer_bwd":
        st["r"], st["c"], st["v"] = _support(case, g)
        st["q"], st["s"] = _encode(_hidden(rows, case["K"], g), fmt)
        st["dy"] = torch.randn(rows, case["M"], device="cuda", generator=g) / rows
        return st
    n = case["n"]
    if op == "norm_fwd":
        st["x"] = torch.randn(rows, n, device="cuda", generator=g) * 0.5
        st["res"] = _hidden(rows, n, g).to(torch.bfloat16 if case["h"] == "bf16" else torch.float32)
        st["gain"] = 1.0 + 0.1 * torch.randn(n, device="cuda", generator=g)
    elif op == "norm_bwd":
        h = _hidden(rows, n, g)
        st["gain"] = 1.0 + 0.1 * torch.randn(n, device="cuda", generator=g)
        st["rstd"] = torch.rsqrt((h * h).mean(-1) + EPS)
        st["dy"] = torch.randn(rows, n, device="cuda", generator=g) / rows
        st["dres"] = torch.randn(rows, n, device="cuda", generator=g) / rows
        if case["h"] in ("int8", "e4m3"):
            st["q"], st["s"] = _encode(h, case["h"])
        else:
            st["hid"] = h.to(torch.bfloat16) if case["h"] == "bf16" else h
    elif op == "pack":
        st["x"] = _hidden(rows, n, g)
    elif op == "gelu_fwd":
        st["x"] = _hidden(rows, n, g, 1.5)
    else:
        st["q"], st["s"] = _encode(_hidden(rows, n, g, 1.5), fmt)
        st["dy"] = torch.randn(rows, n, device="cuda", generator=g) / rows
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        import coo_spmm_amd as L
        fmt = {"f32": L.F32, "bf16": L.BF16, "int8": L.INT8, "e4m3": L.E4M3}
        st["fmt"] = fmt[case["fmt"]]
        if "h" in case:
            st["hfmt"] = fmt[case["h"]]
        if case["op"] == "layer_bwd":     # the layer a training program keeps
            st["layer"] = L.SnackLayer(case["M"], case["K"], st["r"], st["c"], st["v"], seed=1,
                                       max_batch=case["rows"])
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _run_own(st):
    import coo_spmm_amd as L
    case = st["case"]
    op = case["op"]
    if op == "norm_fwd":
        h, y, rstd, ck = L.rmsnorm_fwd(st["x"], st["gain"], EPS, residual=st["res"], q_format=st["fmt"])
        return {"h": h, "y": y, "rstd": rstd, "kept": ck.unpack(torch.bfloat16)}
    if op == "norm_bwd":
        hid = st["hid"] if "hid" in st else L.Ckpt(st["q"], st["s"], st["hfmt"], case["n"])
        dx, dgain = L.rmsnorm_bwd(hid, st["gain"], st["rstd"], st["dy"], dR=st["dres"])
        return {"dx": dx, "dgain": dgain}
    if op == "pack":
        return {"kept": L.Ckpt.pack(st["x"], st["fmt"]).unpack(torch.bfloat16)}
    if op == "gelu_fwd":
        y, cx, cy = L.gelu_ckpt_fwd(st["x"], st["fmt"])
        return {"y": y, "kept_x": cx.unpack(torch.bfloat16), "kept_y": cy.unpack(torch.bfloat16)}
    if op == "gelu_bwd":
        return {"dx": L.gelu_ckpt_bwd(L.Ckpt(st["q"], st["s"], st["fmt"], case["n"]), st["dy"])}
    ck = L.Ckpt(st["q"], st["s"], st["fmt"], case["K"])
    dx, dw = st["layer"].backward_ckpt(ck, st["dy"], want_dx=case["dx"])
    return {"dw": dw, "dx": dx} if case["dx"] else {"dw": dw}


def _cdf(x):
    return 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5)))


def run(st):
    if own:
        return _run_own(st)
    case = st["case"]
    op, fmt = case["op"], case["fmt"]
    if op == "norm_fwd":
        h = (st["x"] + st["res"].float()).to(st["res"].dtype)
        hf = h.float()
        rstd = 1.0 / torch.sqrt((hf * hf).mean(-1) + EPS)
        y = hf * rstd[:, None] * st["gain"]
        return {"h": h, "y": y, "rstd": rstd, "kept": _kept(y, fmt)}
    if op == "norm_bwd":
        h = st["hid"].float() if "hid" in st else _decode(st["q"], st["s"], case["h"], case["n"])
        xh = h * st["rstd"][:, None]
        w = st["dy"] * st["gain"]
        dx = st["rstd"][:, None] * (w - xh * (w * xh).mean(-1, keepdim=True)) + st["dres"]
        return {"dx": dx, "dgain": (st["dy"] * xh).sum(0)}
    if op == "pack":
        return {"kept": _kept(st["x"], fmt)}
    if op == "gelu_fwd":
        y = st["x"] * _cdf(st["x"])
        return {"y": y, "kept_x": _kept(st["x"], fmt), "kept_y": _kept(y, fmt)}
    if op == "gelu_bwd":
        x = _decode(st["q"], st["s"], fmt, case["n"])
        pdf = torch.exp(-0.5 * x * x) * (1.0 / math.sqrt(2.0 * math.pi))
        return {"dx": st["dy"] * (_cdf(x) + x * pdf)}
    r, c = st["r"].long(), st["c"].long()
    x = _decode(st["q"], st["s"], fmt, case["K"])
    out = {"dw": (st["dy"].t() @ x)[r, c]}
    if case["dx"]:
        w = torch.zeros(case["M"], case["K"], device="cuda")
        w[r, c] = st["v"]
        out["dx"] = st["dy"] @ w
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its exact results
# ---------------------------------------------------------------------------

def work(case):
    op, rows = case["op"], case["rows"]
    kept = 1.0 + 1.0 / BLOCK                 # bytes a value takes in a checkpoint
    size = {"f32": 4.0, "bf16": 2.0, "int8": kept, "e4m3": kept}
    if op == "layer_bwd":
        M, K = case["M"], case["K"]
        nnz = M * K * (100 - case["sparsity"]) // 100
        # both passes walk the stored positions: 4 bytes of index each, a value for dX, a dW written
        by = rows * (K * kept + 4.0 * M) + 8.0 * nnz + 4.0 * (M + 1)
        fl = 2.0 * rows * nnz
        if case["dx"]:
            by += 4.0 * rows * K + 4.0 * nnz
            fl *= 2.0
        return {"bytes": by, "flops": fl}
    e = float(rows) * case["n"]
    if op == "norm_fwd":                     # x, residual, h, y, the checkpoint and the values read back from it
        return {"bytes": e * (8.0 + 2.0 * size[case["h"]] + kept + 2.0) + 4.0 * case["n"] + 4.0 * rows, "flops": 6.0 * e}
    if op == "norm_bwd":                     # h, dy, dres, dx
        return {"bytes": e * (12.0 + size[case["h"]]) + 8.0 * case["n"] + 4.0 * rows, "flops": 10.0 * e}
    if op == "pack":
        return {"bytes": e * (4.0 + kept + 2.0), "flops": 3.0 * e}
    if op == "gelu_fwd":                     # x, y, two checkpoints and the values read back from them
        return {"bytes": e * (8.0 + 2.0 * (kept + 2.0)), "flops": 30.0 * e}
    return {"bytes": e * (8.0 + kept), "flops": 40.0 * e}


def _exact_kept(x, fmt):
    """The nearest value of the block's 8-bit grid, in 64 bits."""
    b = _blocks(x)
    top = 127.0 if fmt == "int8" else 448.0
    scale = torch.exp2(torch.ceil(torch.log2(b.abs().amax(-1, keepdim=True) / top)).clamp_min(-126.0))
    v = b / scale
    if fmt == "int8":
        step = torch.ones_like(v)
    else:                                    # 3 fraction bits, smallest step 2^-9
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3.0)
    return (torch.round(v / step) * step * scale).reshape(x.shape[0], -1)[:, :x.shape[1]]


def _exact_decode(q, s, fmt, n):
    """Values from the bytes: sign, exponent and fraction fields (e4m3) or two's complement (int8)."""
    i = q.to(torch.int64)
    if fmt == "int8":
        v = (i - 256 * (i > 127)).double()
    else:
        e, f = (i >> 3) & 15, (i & 7).double()
        v = torch.where(e > 0, (1.0 + f / 8.0) * torch.exp2((e - 7).double()), f * 2.0 ** -9)
        v = torch.where(i > 127, -v, v)
    scale = torch.exp2(s.double() - 127.0)
    return (v * scale.repeat_interleave(BLOCK, dim=1))[:, :n]


def exact(case, seed):
    st = _inputs(case, seed)
    op, fmt = case["op"], case["fmt"]
    if op == "norm_fwd":
        h = (st["x"] + st["res"].float()).to(st["res"].dtype) if case["h"] == "bf16" else None
        hd = h.double() if h is not None else st["x"].double() + st["res"].double()
        rms = torch.sqrt(hd.square().sum(-1) / case["n"] + EPS)
        y = hd / rms[:, None] * st["gain"].double()
        return {"h": hd, "y": y, "rstd": 1.0 / rms, "kept": _exact_kept(y, fmt)}
    if op == "norm_bwd":
        h = st["hid"].double() if "hid" in st else _exact_decode(st["q"], st["s"], case["h"], case["n"])
        r = st["rstd"].double()[:, None]
        dy, gain = st["dy"].double(), st["gain"].double()
        dot = (dy * gain * h).sum(-1, keepdim=True)
        dx = r * dy * gain - r.pow(3) * h * dot / case["n"] + st["dres"].double()
        return {"dx": dx, "dgain": (dy * (h * r)).sum(0)}
    if op == "pack":
        return {"kept": _exact_kept(st["x"].double(), fmt)}
    if op == "gelu_fwd":
        x = st["x"].double()
        y = x * 0.5 * torch.special.erfc(-x / math.sqrt(2.0))
        return {"y": y, "kept_x": _exact_kept(x, fmt), "kept_y": _exact_kept(y, fmt)}
    if op == "gelu_bwd":
        x = _exact_decode(st["q"], st["s"], fmt, case["n"])
        slope = 0.5 * torch.special.erfc(-x / math.sqrt(2.0)) + x * torch.exp(-x * x / 2.0) / math.sqrt(2.0 * math.pi)
        return {"dx": st["dy"].double() * slope}
    # position by position, in pieces that fit
    r, c = st["r"].long(), st["c"].long()
    x = _exact_decode(st["q"], st["s"], fmt, case["K"]).t().contiguous()
    dy = st["dy"].double().t().contiguous()
    piece = max(1, (1 << 26) // case["rows"])
    out = {"dw": torch.cat([(dy[r[i:i + piece]] * x[c[i:i + piece]]).sum(-1) for i in range(0, r.numel(), piece)])}
    if case["dx"]:
        dx = torch.zeros(case["K"], case["rows"], device="cuda", dtype=torch.float64)
        for i in range(0, r.numel(), piece):
            j = slice(i, i + piece)
            dx.index_add_(0, c[j], dy[r[j]] * st["v"].double()[j, None])
        out["dx"] = dx.t()
    return out
