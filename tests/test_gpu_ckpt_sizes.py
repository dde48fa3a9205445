"""The checkpoint operators and the passes under them at sizes where another kernel, variant or launch takes over."""
import numpy as np
import pytest

from snack_inputs import normal, random_layer
from tests import ckpt_oracle as O
from tests.gpu_util import assert_close, dev, host, lib, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,nnz", [(40000, 35000), (9000, 36001)])
@pytest.mark.parametrize("B", [100, 500, 1100])
def test_wide_dw_of_very_short_rows(M, nnz, B):
    """Rows of none, one and a few entries in wide batches: dW on both sides of the choice of entries a wavefront."""
    import oracle
    L = lib()
    K, key = 300, f"sizes/short/{M}/{B}"
    rows, cols, vals = random_layer(M, K, nnz, key)
    layer = L.SnackLayer(M, K, dev(rows), dev(cols), dev(vals), max_batch=B)
    try:
        X, dY = normal((B, K), key + "/x"), normal((B, M), key + "/dy")
        say("short rows", M, nnz, B)
        none, dW = layer.backward(dev(X), dev(dY), want_dx=False)
        r, c, _ = (host(t) for t in layer.export())
        assert none is None and np.bincount(r, minlength=M).min() == 0
        assert_close("dW", host(dW), *oracle.backward_dw(M, K, r, c, X, dY))
    finally:
        layer.close()


def test_plain_calls_need_no_room_for_tiles():
    """The reserve for 64 rows holds the plain passes of 192 here, whose copies are what its partial sums were; only a
    dW from a checkpoint by tiles asks for the tiles' operands too."""
    import oracle
    L = lib()
    M = K = 2500
    nnz, B, key = M * K // 50, 192, "sizes/reserve"
    rows, cols, vals = random_layer(M, K, nnz, key)
    layer = L.SnackLayer(M, K, dev(rows), dev(cols), dev(vals))
    try:
        ref = oracle.canonicalize(M, K, rows, cols, vals)
        X, dY = normal((B, K), key + "/x"), normal((B, M), key + "/dy")
        say("reserve")
        r, c, v = ref["rows"], ref["cols"], ref["vals"]
        assert_close("Y", host(layer.forward(dev(X))), *oracle.forward(M, K, r, c, v, X))
        dX, dW = layer.backward(dev(X), dev(dY))
        assert_close("dX", host(dX), *oracle.backward_dx(M, K, r, c, v, dY))
        assert_close("dW", host(dW), *oracle.backward_dw(M, K, r, c, X, dY))
        ck = L.Ckpt.pack(dev(X), L.INT8)
        dX2, _ = layer.backward_ckpt(ck, dev(dY), want_dw=False)
        assert_close("dX alone", host(dX2), *oracle.backward_dx(M, K, r, c, v, dY))
        with pytest.raises(L.SnackError) as e:
            layer.backward_ckpt(ck, dev(dY))
        assert e.value.code == L.ERR_WORKSPACE
        layer.reserve(B)
        xv = O.unpack(host(ck.q), host(ck.s), O.INT8, K).astype(np.float32)
        dX3, dW3 = layer.backward_ckpt(ck, dev(dY))
        assert_close("dX", host(dX3), *oracle.backward_dx(M, K, r, c, v, dY))
        assert_close("dW", host(dW3), *oracle.backward_dw(M, K, r, c, xv, dY))
    finally:
        layer.close()


@pytest.mark.parametrize("rows,n,last", [((1 << 22) + 70, 3, 100), ((1 << 26) + 5, 4, 100)])
def test_norm_of_more_rows_than_a_launch_takes(rows, n, last):
    """From 2^22 rows of a workgroup each (2^26 of a wavefront) on a launch would pass 2^32 threads: the last rows, and
    those on both sides of the pieces' border, are those of a call on them alone."""
    import torch
    L = lib()
    g = torch.Generator(device="cuda").manual_seed(11)
    x, dr = (torch.randn(rows, n, device="cuda", generator=g) for _ in range(2))
    gain = torch.randn(n, device="cuda", generator=g)
    res = torch.randn(rows, n, device="cuda", generator=g).bfloat16()
    say("many rows", rows, n)
    h, y, rstd, ck = L.rmsnorm_fwd(x, gain, 1e-6, residual=res, q_format=L.E4M3)
    edge = 1 << 21 if n == 3 else 1 << 25
    pieces = [slice(rows - last, rows), slice(edge - 30, edge + 30)]
    kept = []
    for p in pieces:
        h2, y2, r2, c2 = L.rmsnorm_fwd(x[p], gain, 1e-6, residual=res[p], q_format=L.E4M3)
        for a, b in ((h, h2), (y, y2), (rstd, r2), (ck.q, c2.q), (ck.s, c2.s)):
            assert torch.equal(a[p], b)
        kept.append(c2)
    for hid, parts in ((h, [h[p] for p in pieces]), (ck, kept)):
        say("many rows backward", rows, n)
        dx, dg = L.rmsnorm_bwd(hid, gain, rstd, y, dR=dr)
        for p, part in zip(pieces, parts):
            assert torch.equal(dx[p], L.rmsnorm_bwd(part, gain, rstd[p], y[p], dR=dr[p])[0])
        if hid is h:
            # a group adds up its rows' terms in turn, then 8 partial rows a run and 31 runs; 2 roundings of a term
            terms = y.double() * (h.double() * rstd.double()[:, None])
            groups = 256 if n == 3 else 4096     # the sums that are added up in turn: of workgroups, of wavefronts
            tol = (rows // groups + 50) * O.U32 * terms.abs().sum(0)
            assert ((dg.double() - terms.sum(0)).abs() <= tol).all()


def test_norm_of_a_row_longer_than_a_launch():
    """2^27 features: the sum of dgain and the columns of dX in several launches."""
    import torch
    L = lib()
    rows, n, eps = 2, (1 << 27) + 77, 1e-6
    g = torch.Generator(device="cuda").manual_seed(12)
    x, dy = (torch.randn(rows, n, device="cuda", generator=g) for _ in range(2))
    gain = torch.randn(n, device="cuda", generator=g)
    say("long row")
    _, y, rstd, _ = L.rmsnorm_fwd(x, gain, eps)
    xd, gd, dd = x.double(), gain.double(), dy.double()
    rd = ((xd * xd).mean(-1) + float(np.float32(eps))).rsqrt()
    assert ((rstd.double() - rd).abs() <= 1.01 * O.U32 * rd).all()
    want = xd * rd[:, None] * gd
    assert ((y.double() - want).abs() <= 1.01 * O.U32 * want.abs() + 2.0 ** -149).all()
    del want, y
    say("long row backward")
    dx, dg = L.rmsnorm_bwd(x, gain, rstd, dy)
    xh, w = xd * rstd.double()[:, None], dd * gd
    m = (w * xh).mean(-1, keepdim=True)
    # the mean: a thread adds up n / 4096 groups of four in turn, then 6 levels, 16 wavefronts and 6 of a term
    tol = rstd.double()[:, None] * (6 * O.U32 * (w.abs() + (xh * m).abs())
                                    + (n // 4096 + 32) * O.U32 * xh.abs() * (w * xh).abs().mean(-1, keepdim=True))
    assert ((dx.double() - rstd.double()[:, None] * (w - xh * m)).abs() <= tol).all()
    terms = dd * xh
    assert ((dg.double() - terms.sum(0)).abs() <= 4 * O.U32 * terms.abs().sum(0)).all()


@pytest.mark.parametrize("hf", ["f32", "bf16", "int8", "e4m3"])
@pytest.mark.parametrize("rows,n", [(20000, 96), (9000, 700), (3333, 1100), (1500, 4999), (700, 9000), (600, 15001),
                                    (1000, 17001), (3000, 3)])
def test_norm_backward_several_rows_a_workgroup(rows, n, hf):
    """dgain from partial rows of several rows each, in every kernel of the gradient."""
    import torch
    L = lib()
    key = f"sizes/normb/{rows}x{n}"
    x, dy, dr = (normal((rows, n), key + k) for k in ("/h", "/dy", "/dr"))
    gain = (1 + 0.1 * normal((n,), key + "/g")).astype(np.float32)
    rstd = (1 / np.sqrt((x.astype(np.float64) ** 2).mean(-1) + 1e-6)).astype(np.float32)
    if hf in ("int8", "e4m3"):
        h = L.Ckpt.pack(dev(x), O.INT8 if hf == "int8" else O.E4M3)
        hv = host(h.unpack()).astype(np.float64)
    else:
        h = dev(x, torch.bfloat16 if hf == "bf16" else None)
        hv = h.double().cpu().numpy()
    say("several rows", rows, n, hf)
    dx, dg = L.rmsnorm_bwd(h, dev(gain), dev(rstd), dev(dy), dev(dr))
    dxr, dgr, ax, ag = O.norm_bwd(hv, gain, rstd, dy, dr)
    # the mean: at most 20 features a thread, 6 levels, 16 wavefronts, 3 of a term; 6 more to dx
    assert (np.abs(host(dx) - dxr) <= 51 * O.U32 * ax).all()
    # a unit's rows in turn (256 units at least), 3 wavefronts, 1024 / 32 partial rows in turn, 31 runs, 2 of a term
    tol = (-(-rows // 256) + 3 + 32 + 31 + 2) * O.U32 * ag
    assert (np.abs(host(dg) - dgr) <= tol).all()


def test_norm_dgain_of_many_rows():
    """Over a thousand rows a workgroup, against the column sums in 64 bits."""
    import torch
    L = lib()
    rows, n = 400000, 1500
    g = torch.Generator(device="cuda").manual_seed(13)
    x, dy = (torch.randn(rows, n, device="cuda", generator=g) for _ in range(2))
    gain, rstd = torch.randn(n, device="cuda", generator=g), torch.rand(rows, device="cuda", generator=g) + 0.5
    ck = L.Ckpt.pack(x, L.INT8)
    for h, hv in ((x, x), (ck, ck.unpack())):
        say("many rows dgain")
        _, dg = L.rmsnorm_bwd(h, gain, rstd, dy)
        want, mag = torch.zeros(n, device="cuda", dtype=torch.float64), torch.zeros(n, device="cuda", dtype=torch.float64)
        for a in range(0, rows, 50000):
            t = dy[a:a + 50000].double() * (hv[a:a + 50000].double() * rstd[a:a + 50000].double()[:, None])
            want += t.sum(0)
            mag += t.abs().sum(0)
        assert ((dg.double() - want).abs() <= (-(-rows // 256) + 68) * O.U32 * mag).all()


@pytest.mark.parametrize("M,K,nnz", [(2000, 2000, 200000), (1050, 3200, 168000), (1050, 3200, 60000)])
def test_layer_gradients_two_wavefronts_a_tile(M, K, nnz):
    """Layers of 1008 and of 825 tiles: two tiles a workgroup, and an odd one left; batches below a step a wavefront."""
    from tests.test_gpu_ckpt import _layer_case
    _layer_case(M, K, nnz, (8, 16, 33, 100), f"sizes/two/{M}x{K}/{nnz}", [O.INT8])


@pytest.mark.parametrize("power", [-109, -118, -126])
def test_layer_dw_of_tiny_gradients(power):
    """dY's three parts are exact from 2^-109 on; below that the last ends at steps of 2^-133, so a term may lose less
    than that times its x."""
    L = lib()
    M, K, nnz, B, key = 300, 260, 12000, 64, "sizes/tiny"
    rows, cols, vals = random_layer(M, K, nnz, key)
    layer = L.SnackLayer(M, K, dev(rows), dev(cols), dev(vals))
    try:
        dY = normal((B, M), key + "/dy")
        dY = (np.sign(dY) * (1 + np.abs(dY) % 1) * 2.0 ** power).astype(np.float32)
        ck = L.Ckpt.pack(dev(normal((B, K), key + "/x") * 4096), O.INT8)
        say("tiny", power)
        _, dW = layer.backward_ckpt(ck, dev(dY), want_dx=False)
        r, c, _ = (host(t) for t in layer.export())
        xv, d = host(ck.unpack()).astype(np.float64), dY.astype(np.float64)
        want, mag = (d[:, r] * xv[:, c]).sum(0), (np.abs(d[:, r]) * np.abs(xv[:, c])).sum(0)
        # 3 B additions in fp32 and the steps in which they end
        tol = 3 * B * (O.U32 * mag + 2.0 ** -150) + (0 if power >= -109 else 2.0 ** -133 * np.abs(xv[:, c]).sum(0))
        assert (np.abs(host(dW) - want) <= tol).all(), np.abs(host(dW) - want).max() / mag.max()
    finally:
        layer.close()


def test_layer_dw_operands_past_two_gb():
    """The tiles' operands lie at 32-bit offsets of a scalar base: dY's take 2.4 GB here."""
    import torch
    L = lib()
    M, K, B, key = 10000, 1000, 40000, "sizes/operands"
    nnz = M * K // 32
    rows, cols, vals = random_layer(M, K, nnz, key)
    g = torch.Generator(device="cuda").manual_seed(14)
    X, dY = torch.randn(B, K, device="cuda", generator=g), torch.randn(B, M, device="cuda", generator=g)
    layer = L.SnackLayer(M, K, dev(rows), dev(cols), dev(vals), max_batch=B)
    try:
        ck = L.Ckpt.pack(X, L.E4M3)
        say("operands", M, K, B)
        _, dW = layer.backward_ckpt(ck, dY, want_dx=False)
        r, c, _ = layer.export()
        xv = ck.unpack()
        for i in (0, nnz // 2, nnz - 1500):
            k = slice(i, i + 1500)
            a, b = dY[:, r[k].long()].double(), xv[:, c[k].long()].double()
            tol = 3 * B * O.U32 * (a.abs() * b.abs()).sum(0)
            assert ((dW[k].double() - (a * b).sum(0)).abs() <= tol).all()
    finally:
        layer.close()
        torch.cuda.empty_cache()
