"""Activation checkpoints, the residual norm, the GELU and the layer's gradients from a checkpoint, against 64-bit
references.  Tolerances are sums of the roundings (u = 2^-24, half a step of fp32, relative) along the longest chain."""
import numpy as np
import pytest

from snack_inputs import normal, random_layer
from tests import ckpt_oracle as O
from tests.gpu_util import assert_close, dev, host, lib, say

pytestmark = pytest.mark.gpu

FMTS = [O.INT8, O.E4M3]
# widths: one feature, inside a block, a block, ragged, one wavefront's longest row and one past it, a workgroup's
# longest and one past it
SHAPES = [(1, 1), (3, 31), (2, 32), (5, 33), (7, 77), (1, 768), (65, 500), (6, 1024), (5, 1025), (9, 4999),
          (3, 16384), (2, 16385)]


def _x(rows, n, key, spread=True):
    x = normal((rows, n), key)
    x[:, ::17] *= 8.0
    if spread:   # rows of very different magnitude, one of them all zeros
        x *= np.exp2((np.arange(rows) * 13 % 61 - 30).astype(np.float32))[:, None]
        if rows > 2:
            x[2] = 0.0
    return x.astype(np.float32)


def _same(got, want, what):
    bad = np.argwhere(got != want)
    assert bad.size == 0, f"{what}: {bad.shape[0]} differ, first at {bad[0]}: {got[tuple(bad[0])]} {want[tuple(bad[0])]}"


def _close(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first at {i}: {got[i]} for {want[i]}, "
                             f"tolerance {np.broadcast_to(tol, bad.shape)[i]}")


def _misaligned(a):
    """The array on the device, its base four bytes past a 16-byte boundary."""
    import torch
    flat = torch.empty(a.size + 1, device="cuda", dtype=torch.float32)
    t = flat[1:].view(a.shape)
    t.copy_(torch.from_numpy(np.ascontiguousarray(a)))
    assert t.data_ptr() % 16 == 4
    return t


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,n", SHAPES)
def test_pack_and_unpack_are_exact(rows, n, fmt):
    import torch
    L = lib()
    x = _x(rows, n, f"ckpt/pack/{rows}x{n}")
    say("pack", rows, n, fmt)
    for t in (dev(x), _misaligned(x)):
        ck = L.Ckpt.pack(t, fmt)
        q, s = O.pack(x, fmt)
        _same(host(ck.s), s, "exponents")
        _same(host(ck.q), q, "codes")
    v = O.unpack(q, s, fmt, n)
    _same(host(ck.unpack()).astype(np.float64), v, "fp32 values")
    _same(host(ck.unpack(torch.bfloat16).float()).astype(np.float64), v, "bf16 values")
    assert ck.nbytes == rows * 33 * (-(-n // 32))


@pytest.mark.parametrize("fmt", FMTS)
def test_pack_borders(fmt):
    """Largest values on both sides of every border: of the format's range, of fp32's, halfway codes, and blocks
    with a NaN or an infinity, whose neighbours stay as they are."""
    L = lib()
    top = 127.0 if fmt == O.INT8 else 448.0
    x = np.zeros((12, 64), np.float32)
    half = np.array([k + 0.5 for k in range(32)], np.float32)
    x[0, :32] = half
    x[0, 0] = top
    x[1, 0], x[1, 1] = np.nextafter(np.float32(top), np.float32(1e9)), 1.0
    x[2, 0] = np.nextafter(np.float32(top), np.float32(0))
    x[3, 0], x[3, 1] = np.finfo(np.float32).max, -1e30
    x[4, 0], x[4, 5] = np.finfo(np.float32).tiny, 1e-45
    x[5, 0], x[5, 1] = 1e-45, -1e-40
    x[6, 3], x[6, 40] = np.inf, 2.0
    x[7, 3], x[7, 40] = np.nan, 2.0
    x[8, 35], x[8, 1] = -np.inf, 2.0
    x[9, 0], x[9, 1:20] = top, np.linspace(2.0 ** -11, 2.0 ** -6, 19)
    x[10, 0] = -0.0
    x[11] = np.linspace(-top, top, 64)
    say("pack borders", fmt)
    ck = L.Ckpt.pack(dev(x), fmt)
    q, s = O.pack(x, fmt)
    _same(host(ck.s), s, "exponents")
    if fmt == O.INT8:
        _same(host(ck.q), q, "codes")
    else:   # the sign of a zero code is free
        _same(host(ck.q) & np.where(q & 127, 255, 127), q & np.where(q & 127, 255, 127), "codes")
    got = host(ck.unpack())
    with np.errstate(over="ignore"):
        want = O.unpack(q, s, fmt, 64).astype(np.float32)    # fp32's largest rounds up to 2^128: infinity in fp32
    assert np.isinf(want[3, 0]) and np.array_equal(got, want, equal_nan=True)
    assert np.isnan(got[6, :32]).all() and got[6, 40] == 2.0 and got[8, 1] == 2.0


@pytest.mark.parametrize("fmt", FMTS)
def test_unpack_any_bytes(fmt):
    """Every code under every exponent byte, 0 and 255 among them; bytes past the row's end are not read as values."""
    import torch
    L = lib()
    q = np.tile(np.arange(256, dtype=np.uint8), (256, 1)).reshape(2048, 32)
    s = np.repeat(np.arange(256, dtype=np.uint8), 8).reshape(2048, 1)
    say("unpack any", fmt)
    ck = L.Ckpt(dev(q), dev(s), fmt, 32)
    want = O.unpack(q, s, fmt, 32)
    with np.errstate(over="ignore"):
        w32 = want.astype(np.float32)
    assert np.array_equal(host(ck.unpack()), w32, equal_nan=True)
    wb = torch.from_numpy(w32).to(torch.bfloat16).float().numpy()
    assert np.array_equal(host(ck.unpack(torch.bfloat16).float()), wb, equal_nan=True)
    short = L.Ckpt(dev(q), dev(s), fmt, 27)
    assert np.array_equal(host(short.unpack()), w32[:, :27], equal_nan=True)


def _norm_case(rows, n, hf, key):
    import torch
    x = _x(rows, n, key + "/x", spread=False)
    res = _x(rows, n, key + "/r", spread=False) * 3
    if rows > 2:
        x[2] = 0.0
        res[2] = 0.0          # a row of zeros: rstd = 1 / sqrt(eps)
    gain = (1 + 0.1 * normal((n,), key + "/g")).astype(np.float32)
    rt = dev(res, torch.bfloat16 if hf == "bf16" else torch.float32)
    h = (torch.from_numpy(x) + rt.float().cpu()).to(rt.dtype)      # the definition's one rounding (and bf16's)
    return x, rt, gain, h


@pytest.mark.parametrize("hf", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n", SHAPES)
def test_norm_forward(rows, n, hf):
    import torch
    L = lib()
    x, rt, gain, h = _norm_case(rows, n, hf, f"norm/{rows}x{n}")
    eps = 1e-6
    for fmt in FMTS:
        say("norm fwd", rows, n, hf, fmt)
        H, y, rstd, ck = L.rmsnorm_fwd(dev(x), dev(gain), eps, residual=rt, q_format=fmt)
        assert H.dtype == rt.dtype and torch.equal(H.cpu(), h)
        yr, rr = O.norm_fwd(h.float().numpy(), gain, np.float64(np.float32(eps)))
        # the sum: 16 squares a thread, 6 levels, 16 wavefronts (rows past 16384: 8 more groups): under 56
        # roundings, halved by the root; then mean, eps, root and quotient
        _close(host(rstd), rr, 34 * O.U32 * rr, "rstd")
        _close(host(y), yr, 37 * O.U32 * np.abs(yr), "y")
        q, s = O.pack(host(y), fmt)
        _same(host(ck.s), s, "exponents")
        _same(host(ck.q), q, "codes")
        _, none, rstd2, ck2 = L.rmsnorm_fwd(dev(x), dev(gain), eps, residual=rt, q_format=fmt, want_y=False)
        assert none is None and torch.equal(ck2.q, ck.q) and torch.equal(ck2.s, ck.s) and torch.equal(rstd2, rstd)
    xt = _misaligned(x)
    hx, y, _, ck = L.rmsnorm_fwd(xt, dev(gain), eps)
    assert hx is xt and ck is None
    yr, _ = O.norm_fwd(x, gain, np.float64(np.float32(eps)))
    _close(host(y), yr, 37 * O.U32 * np.abs(yr), "y without residual")


@pytest.mark.parametrize("rows,n", [(8000, 4999), (2400, 17001), (44000, 900)])
def test_norm_forward_large(rows, n):
    """Outputs past the caches are stored another way: the same bits as in pieces that are not."""
    import torch
    L = lib()
    g = torch.Generator(device="cuda").manual_seed(8)
    x, gain = torch.randn(rows, n, device="cuda", generator=g), torch.randn(n, device="cuda", generator=g)
    res = torch.randn(rows, n, device="cuda", generator=g).bfloat16()
    say("norm large", rows, n)
    h, y, rstd, ck = L.rmsnorm_fwd(x, gain, 1e-6, residual=res, q_format=L.E4M3)
    assert rows * n * 7 > 256 << 20
    for a in range(0, rows, 1000):
        b = min(rows, a + 1000)
        h2, y2, r2, c2 = L.rmsnorm_fwd(x[a:b], gain, 1e-6, residual=res[a:b], q_format=L.E4M3)
        for t, u in ((h, h2), (y, y2), (rstd, r2), (ck.q, c2.q), (ck.s, c2.s)):
            assert torch.equal(t[a:b], u), a


@pytest.mark.parametrize("hf", ["f32", "bf16", "int8", "e4m3"])
@pytest.mark.parametrize("rows,n", SHAPES + [(2100, 96), (600, 1100)])
def test_norm_backward(rows, n, hf):
    import torch
    L = lib()
    key = f"normb/{rows}x{n}"
    x = _x(rows, n, key + "/h", spread=False)
    gain = (1 + 0.1 * normal((n,), key + "/g")).astype(np.float32)
    rstd = (1 / np.sqrt((x.astype(np.float64) ** 2).mean(-1) + 1e-6)).astype(np.float32)
    dy, dr = normal((rows, n), key + "/dy"), normal((rows, n), key + "/dr")
    if hf in ("int8", "e4m3"):
        q, s = O.pack(x, O.INT8 if hf == "int8" else O.E4M3)
        hv = O.unpack(q, s, O.INT8 if hf == "int8" else O.E4M3, n)
        if n % 32:       # bytes past the row's end must not matter: NaN codes and the largest integers
            q.reshape(rows, -1)[:, n:] = 0x7F
        h = L.Ckpt(dev(q), dev(s), O.INT8 if hf == "int8" else O.E4M3, n)
    else:
        h = dev(x, torch.bfloat16 if hf == "bf16" else torch.float32)
        hv = h.double().cpu().numpy()
    for with_dr in (True, False):
        say("norm bwd", rows, n, hf, with_dr)
        r = dr if with_dr else None
        dx, dg = L.rmsnorm_bwd(h, dev(gain), dev(rstd), dev(dy), dev(dr) if with_dr else None)
        dxr, dgr, ax, ag = O.norm_bwd(hv, gain, rstd, dy, r)
        # mean: under 56 roundings of the sum and 3 of each term; 6 more to dx
        _close(host(dx), dxr, 65 * O.U32 * ax, "dx")
        # dgain: up to 5 rows a wavefront, 3 wavefronts, 16 partial rows in turn and 31 runs, 3 of a term
        _close(host(dg), dgr, 60 * O.U32 * ag + 1e-30, "dgain")
    dx2, none = L.rmsnorm_bwd(h, dev(gain), dev(rstd), dev(dy), want_dgain=False)
    assert none is None and torch.equal(dx2, dx)
    again = L.rmsnorm_bwd(h, dev(gain), dev(rstd), dev(dy))
    assert torch.equal(again[0], dx) and torch.equal(again[1], dg)


def test_past_two_to_the_31():
    """Arrays of more than 2^31 values: the last rows are those of a call on them alone."""
    import torch
    L = lib()
    rows, n, last = 214800, 10007, 70
    assert rows * n > 2 ** 31 and torch.cuda.mem_get_info()[0] > 80e9
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(rows, n, device="cuda", generator=g)
    gain = torch.randn(n, device="cuda", generator=g)
    tail = x[rows - last:].clone()
    try:
        say("large pack")
        ck, ct = L.Ckpt.pack(x, L.INT8), L.Ckpt.pack(tail, L.INT8)
        assert torch.equal(ck.q[rows - last:], ct.q) and torch.equal(ck.s[rows - last:], ct.s)
        for dt in (torch.float32, torch.bfloat16):
            say("large unpack", dt)
            assert torch.equal(ck.unpack(dt)[rows - last:], ct.unpack(dt))
        say("large norm")
        h, y, rstd, cy = L.rmsnorm_fwd(x, gain, 1e-6, residual=x, q_format=L.E4M3)
        ht, yt, rt, cyt = L.rmsnorm_fwd(tail, gain, 1e-6, residual=tail, q_format=L.E4M3)
        for a, b in ((h, ht), (y, yt), (rstd, rt), (cy.q, cyt.q), (cy.s, cyt.s)):
            assert torch.equal(a[rows - last:], b)
        del h, cy
        say("large norm backward")
        for hid, hid_t in ((x, tail), (ck, ct)):
            dx, dg = L.rmsnorm_bwd(hid, gain, rstd, y, dR=x)
            dxt, _ = L.rmsnorm_bwd(hid_t, gain, rt, yt, dR=tail)
            assert torch.equal(dx[rows - last:], dxt) and bool(torch.isfinite(dg).all())
            del dx
        say("large gelu")
        assert torch.equal(L.gelu_ckpt_bwd(ck, y)[rows - last:], L.gelu_ckpt_bwd(ct, yt))
        a, cx, ca = L.gelu_ckpt_fwd(x, L.E4M3)
        at, cxt, cat = L.gelu_ckpt_fwd(tail, L.E4M3)
        for u, v in ((a, at), (cx.q, cxt.q), (ca.q, cat.q), (ca.s, cat.s)):
            assert torch.equal(u[rows - last:], v)
    finally:
        x = y = a = None
        torch.cuda.empty_cache()


@pytest.mark.parametrize("rows,n", [(1, 1), (5, 33), (64, 500), (3, 4999), (130, 3100)])
def test_gelu_checkpointed(rows, n):
    import torch
    L = lib()
    x = (_x(rows, n, f"gelu/{rows}x{n}", spread=False) * 1.5).astype(np.float32)
    x.flat[: min(x.size, 40)] = np.linspace(-20, 20, 40, dtype=np.float32)[: min(x.size, 40)]
    dy = normal((rows, n), f"gelu/{rows}x{n}/dy")
    for fmt in FMTS:
        say("gelu", rows, n, fmt)
        y, cx, cy = L.gelu_ckpt_fwd(dev(x), fmt)
        # Phi: 3.2e-8 of the polynomial and nine roundings of R, e and their product, each on at most 1/2;
        # 1 - q and the product with x one more each
        _close(host(y), O.gelu(x), 6 * O.U32 * np.abs(x) + 1e-37, "y")
        for ck, v in ((cx, x), (cy, host(y))):
            q, s = O.pack(v, fmt)
            _same(host(ck.s), s, "exponents")
            _same(host(ck.q) & np.where(q & 127, 255, 127), q & np.where(q & 127, 255, 127), "codes")
        none, cx2, cy2 = L.gelu_ckpt_fwd(dev(x), fmt, want_y=False)
        assert none is None and torch.equal(cx2.q, cx.q) and torch.equal(cy2.q, cy.q) and torch.equal(cy2.s, cy.s)
        xv = O.unpack(*O.pack(x, fmt), fmt, n)
        dx = L.gelu_ckpt_bwd(cx, dev(dy))
        _close(host(dx), dy * O.gelu_slope(xv), 6 * O.U32 * np.abs(dy) + 1e-37, "dx")


def test_gelu_non_finite():
    L = lib()
    x = np.zeros((1, 64), np.float32)
    x[0, :3] = [np.inf, -20.0, np.nan]
    y, _, cy = L.gelu_ckpt_fwd(dev(x), O.INT8)
    g = host(y)
    assert g[0, 0] == np.inf and g[0, 1] <= 0 and abs(g[0, 1]) < 1e-37 and np.isnan(g[0, 2])
    v = host(cy.unpack())
    assert np.isnan(v[0, :32]).all() and (v[0, 32:] == 0).all()
    q = np.zeros((1, 32), np.uint8)
    q[0, :2] = [1, 255]                                       # +inf, -inf under exponent byte 255; 0 gives NaN
    ck = L.Ckpt(dev(q), dev(np.full((1, 1), 255, np.uint8)), O.INT8, 32)
    d = host(L.gelu_ckpt_bwd(ck, dev(np.ones((1, 32), np.float32))))
    assert d[0, 0] == 1.0 and d[0, 1] == 0.0 and np.isnan(d[0, 2:]).all()


LAYERS = [(1, 1, 1), (1, 300, 17), (300, 1, 29), (7, 9, 0), (37, 53, 400), (130, 70, 2000), (257, 129, 33153),
          (64, 4096, 20000), (700, 500, 35000), (513, 1500, 76000)]


def _layer_case(M, K, nnz, batches, key, fmts=FMTS, triple=None):
    """dX and dW, together and alone, against the sums in 64 bits."""
    import oracle
    import torch
    L = lib()
    rows, cols, vals = triple if triple is not None else random_layer(M, K, nnz, key)
    ref = oracle.canonicalize(M, K, rows, cols, vals)
    layer = L.SnackLayer(M, K, dev(rows), dev(cols), dev(vals), max_batch=max(batches))
    try:
        for B in batches:
            dY = normal((B, M), f"{key}/dY/{B}")
            X = normal((B, K), f"{key}/X/{B}") * np.exp2(np.arange(B) % 7 - 3).astype(np.float32)[:, None]
            for fmt in fmts:
                say("layer", key, "B", B, fmt)
                ck = L.Ckpt.pack(dev(X), fmt)
                xv = O.unpack(host(ck.q), host(ck.s), fmt, K).astype(np.float32)
                dX, dW = layer.backward_ckpt(ck, dev(dY))
                dXr, dXa = oracle.backward_dx(M, K, ref["rows"], ref["cols"], ref["vals"], dY)
                assert_close(f"dX B={B}", host(dX), dXr, dXa)
                dWr, dWa = oracle.backward_dw(M, K, ref["rows"], ref["cols"], xv, dY)
                assert_close(f"dW B={B}", host(dW), dWr, dWa)
                none, dW2 = layer.backward_ckpt(ck, dev(dY), want_dx=False)
                assert none is None
                assert_close(f"dW alone B={B}", host(dW2), dWr, dWa)
                dX2, none = layer.backward_ckpt(ck, dev(dY), want_dw=False)
                assert none is None
                assert_close(f"dX alone B={B}", host(dX2), dXr, dXa)
                again = layer.backward_ckpt(ck, dev(dY))
                assert torch.equal(again[0], dX) and torch.equal(again[1], dW)
    finally:
        layer.close()


@pytest.mark.parametrize("M,K,nnz", LAYERS)
def test_layer_gradients(M, K, nnz):
    _layer_case(M, K, nnz, (1, 2, 3, 5, 8, 13, 17, 33, 64, 65, 130), f"ckpt/layer/{M}x{K}/{nnz}")


def test_layer_gradients_wide():
    _layer_case(3072, 768, 235929, (1024,), "ckpt/layer/up", [O.INT8])
    _layer_case(768, 3072, 23592, (1000,), "ckpt/layer/down", [O.E4M3])


@pytest.mark.parametrize("M,K,nnz", [(6000, 900, 540000), (4100, 1200, 100000), (40, 32640, 45000), (40, 32641, 45000)])
def test_layer_gradients_many_tiles(M, K, nnz):
    """A wavefront a tile; long and short lists of a tile; the widest layer with tiles and one past it."""
    _layer_case(M, K, nnz, (8, 33, 100), f"ckpt/tiles/{M}x{K}", [O.INT8])


def test_layer_gradients_short_rows():
    """Wide batches over rows of about a dozen positions: runs of four that lie in one row, that do not, and a tail."""
    _layer_case(3000, 900, 35003, (65, 300), "ckpt/short", [O.E4M3])


def test_captured_gradient_reads_the_present_index():
    """A call captured before a drop/regrow and replayed after it."""
    import torch
    L = lib()
    M, K, nnz, B, key = 300, 260, 12000, 64, "ckpt/captured"
    rows, cols, vals = random_layer(M, K, nnz, key)
    layer = L.SnackLayer(M, K, dev(rows), dev(cols), dev(vals), seed=4)
    try:
        ck, dY = L.Ckpt.pack(dev(normal((B, K), key + "/x")), L.E4M3), dev(normal((B, M), key + "/dy"))
        dW = torch.zeros(nnz, device="cuda")
        graphs = []
        for warm in (False, True):       # captured as the layer's first such call, and after an eager one
            say("capture", warm)
            if warm:
                layer.backward_ckpt(ck, dY, want_dx=False, dW=dW)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                layer.backward_ckpt(ck, dY, want_dx=False, dW=dW)
            graphs.append(g)
        for step in range(3):
            for i, g in enumerate(graphs):
                say("replay", step, i)
                dW.zero_()
                g.replay()
                torch.cuda.synchronize()
                assert torch.equal(dW, layer.backward_ckpt(ck, dY, want_dx=False)[1])
            layer.prune_regrow(3000)
    finally:
        layer.close()


def test_layer_gradients_follow_the_support():
    """After drop/regrow and a value change the gradients are those of the new triple."""
    import oracle
    L = lib()
    M, K, nnz, key = 300, 260, 12000, "ckpt/regrow"
    rows, cols, vals = random_layer(M, K, nnz, key)
    layer = L.SnackLayer(M, K, dev(rows), dev(cols), dev(vals), seed=3, max_batch=130)
    try:
        for step in range(3):
            for B in (4, 64, 130):
                X, dY = normal((B, K), f"{key}/X/{step}/{B}"), normal((B, M), f"{key}/dY/{step}/{B}")
                ck = L.Ckpt.pack(dev(X), O.INT8)
                xv = O.unpack(host(ck.q), host(ck.s), O.INT8, K).astype(np.float32)
                say("regrow", step, B)
                dX, dW = layer.backward_ckpt(ck, dev(dY))
                r, c, v = (host(t) for t in layer.export())
                assert_close("dX", host(dX), *oracle.backward_dx(M, K, r, c, v, dY))
                assert_close("dW", host(dW), *oracle.backward_dw(M, K, r, c, xv, dY))
                layer.sgd_step(dW, 0.01)
            layer.prune_regrow(3000)
    finally:
        layer.close()


@pytest.mark.parametrize("how", ["random", "gradient", "rows"])
def test_layer_gradients_after_every_regrow(how):
    """The tile list follows each kind of drop/regrow."""
    import oracle
    L = lib()
    M, K, nnz, B, key = 150, 400, 6000, 70, "ckpt/kinds"
    rows, cols, vals = random_layer(M, K, nnz, key)
    layer = L.SnackLayer(M, K, dev(rows), dev(cols), dev(vals), seed=5, max_batch=B)
    try:
        X, dY = normal((B, K), key + "/X"), normal((B, M), key + "/dY")
        ck = L.Ckpt.pack(dev(X), O.INT8)
        xv = O.unpack(host(ck.q), host(ck.s), O.INT8, K).astype(np.float32)
        for step in range(3):
            say("kinds", how, step)
            dX, dW = layer.backward_ckpt(ck, dev(dY))
            r, c, v = (host(t) for t in layer.export())
            assert_close("dX", host(dX), *oracle.backward_dx(M, K, r, c, v, dY))
            assert_close("dW", host(dW), *oracle.backward_dw(M, K, r, c, xv, dY))
            if how == "random":
                layer.prune_regrow(1500)
            elif how == "gradient":
                layer.prune_regrow_grad(1500, dev(X), dev(dY))
            else:
                layer.prune_regrow_rows(1, 4)
    finally:
        layer.close()


@pytest.mark.parametrize("B", [3, 20, 64, 130])
def test_layer_gradients_non_finite(B):
    """A NaN or an infinity of dY reaches its own row's dW, one of x its own column's; the rest is as without."""
    import oracle
    L = lib()
    M, K, nnz, key = 150, 200, 6000, "ckpt/nonfinite"
    rows, cols, vals = random_layer(M, K, nnz, key)
    layer = L.SnackLayer(M, K, dev(rows), dev(cols), dev(vals), max_batch=B)
    try:
        X, dY = normal((B, K), f"{key}/X/{B}"), normal((B, M), f"{key}/dY/{B}")
        X[0, 40] = np.nan                                 # its block of 32 columns reads as NaN
        clean = L.Ckpt.pack(dev(np.nan_to_num(X)), O.E4M3)
        xv = O.unpack(host(clean.q), host(clean.s), O.E4M3, K).astype(np.float32)
        r, c, _ = (host(t) for t in layer.export())
        want, mag = oracle.backward_dw(M, K, r, c, xv, dY)
        dY[1, 7], dY[2, 9] = np.nan, np.inf
        ck = L.Ckpt.pack(dev(X), O.E4M3)
        bad = (r == 7) | (r == 9) | ((c >= 32) & (c < 64))
        for want_dx in (False, True):
            say("non finite", B, want_dx)
            dW = host(layer.backward_ckpt(ck, dev(dY), want_dx=want_dx)[1])
            assert not np.isfinite(dW[bad]).any()
            assert_close("dW", dW[~bad], want[~bad], mag[~bad])
    finally:
        layer.close()


def test_layer_refusals_leave_outputs():
    import torch
    L = lib()
    M, K = 200, 150
    rows, cols, vals = random_layer(M, K, 3000, "ckpt/refuse")
    layer = L.SnackLayer(M, K, dev(rows), dev(cols), dev(vals))
    try:
        ck = L.Ckpt.pack(dev(normal((200, K), "ckpt/refuse/x")), L.INT8)
        dY = dev(normal((200, M), "ckpt/refuse/dy"))
        dX, dW = torch.full((200, K), 7.0, device="cuda"), torch.full((3000,), 7.0, device="cuda")
        with pytest.raises(L.SnackError) as e:      # the reserve covers batches up to 64
            layer.backward_ckpt(ck, dY, dX=dX, dW=dW)
        assert e.value.code == L.ERR_WORKSPACE
        assert bool((dX == 7).all()) and bool((dW == 7).all())
        with pytest.raises(ValueError):
            layer.backward_ckpt(ck, dY[:, :-1].contiguous())
        with pytest.raises(ValueError):
            layer.backward_ckpt(L.Ckpt.pack(dY, L.INT8), dY)
        with pytest.raises(TypeError):
            layer.backward_ckpt(ck, dY.double())
        with pytest.raises(ValueError):
            L.rmsnorm_fwd(dY, dev(np.ones(M + 1, np.float32)), 1e-6)
        with pytest.raises(ValueError):
            L.Ckpt.pack(dY.t(), L.INT8)
    finally:
        layer.close()


def test_no_rows():
    import torch
    L = lib()
    x, g = torch.empty(0, 40, device="cuda"), torch.ones(40, device="cuda")
    h, y, rstd, ck = L.rmsnorm_fwd(x, g, 1e-6, residual=x.bfloat16(), q_format=L.INT8)
    assert h.shape == (0, 40) and y.shape == (0, 40) and rstd.shape == (0,) and ck.rows == 0
    dx, dg = L.rmsnorm_bwd(ck, g, rstd, x)
    assert dx.shape == (0, 40) and bool((dg == 0).all())
    assert ck.unpack().shape == (0, 40)
    assert L.gelu_ckpt_bwd(L.gelu_ckpt_fwd(x, L.E4M3)[1], x).shape == (0, 40)


def test_other_stream_and_graph():
    """On a stream of its own, and replayed from a graph with other work between the replays."""
    import torch
    L = lib()
    M, K, B = 300, 260, 130
    rows, cols, vals = random_layer(M, K, 9000, "ckpt/graph")
    layer = L.SnackLayer(M, K, dev(rows), dev(cols), dev(vals), max_batch=B)
    try:
        g = dev((1 + 0.1 * normal((K,), "ckpt/graph/g")).astype(np.float32))
        x, dY = dev(normal((B, K), "ckpt/graph/x")), dev(normal((B, M), "ckpt/graph/dy"))

        def step(stream=None):
            h, y, rstd, ck = L.rmsnorm_fwd(x, g, 1e-6, residual=x, q_format=L.INT8, stream=stream)
            dX, dW = layer.backward_ckpt(ck, dY, stream=stream)
            dh, dg = L.rmsnorm_bwd(h, g, rstd, dX, dR=dX, stream=stream)
            a, cx, cy = L.gelu_ckpt_fwd(dh, L.E4M3, stream=stream)
            return y, dX, dW, dh, dg, a, cy.unpack(stream=stream), L.gelu_ckpt_bwd(cx, a, stream=stream)

        say("eager")
        want = [t.clone() for t in step()]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        say("stream")
        got = step(s)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        say("graph")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step()
        for i in range(4):
            for o in outs:
                o.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want)), i
            step()
    finally:
        layer.close()
