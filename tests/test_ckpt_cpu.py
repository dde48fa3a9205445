"""The checkpoint operators without a GPU: the oracle's format against torch's own e4m3 and closed forms, the
norm's and the GELU's gradients against differences, and every refusal that is decided on the host."""
import ctypes
import os

import numpy as np
import pytest

from tests import ckpt_oracle as O


def _lib():
    import coo_spmm_amd as L
    if not os.path.exists(L.LIB_PATH):
        import __graft_entry__
        __graft_entry__._builder().build()
    return L


def test_oracle_e4m3_codes_match_torch():
    import torch
    c = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(c).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(np.nan_to_num(t, nan=1e9), np.nan_to_num(O.e4m3_table(), nan=1e9))


@pytest.mark.parametrize("fmt", [O.INT8, O.E4M3])
def test_oracle_pack_properties(fmt):
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((9, 77)) * np.exp2(rng.integers(-40, 40, (9, 1)))).astype(np.float32)
    x[3] = 0
    x[4, :32] = 127.0
    x[5, :32] = 448.0
    x[6, 40] = np.inf
    x[7, 76] = np.nan
    q, s = O.pack(x, fmt)
    assert (q.reshape(9, 3, 32)[:, 2, 13:] == 0).all()
    assert (s[3] == 1).all() and s[6, 1] == 255 and s[7, 2] == 255 and s[6, 0] != 255
    if fmt == O.INT8:
        assert s[4, 0] == 127 and s[5, 0] == 129      # 127 = 127 * 2^0; 448 = 112 * 2^2
    else:
        assert s[4, 0] == 126 and s[5, 0] == 127      # 127 <= 448 / 2; 448 = 448 * 2^0
    y = O.unpack(q, s, fmt, 77)
    good = np.isfinite(y)
    assert np.isnan(y[6, 32:64]).all() and np.isnan(y[7, 64:]).all() and good[:6].all()
    # half a step: of the block's grid (int8), of the value or of the smallest code (e4m3)
    sc = np.repeat(np.exp2(s.astype(np.float64) - 127), 32, 1)[:, :77]
    bound = sc * 0.5 if fmt == O.INT8 else np.maximum(np.abs(x) * 2.0 ** -4, sc * 2.0 ** -10)
    assert (np.abs(y - x)[good] <= bound[good]).all()
    if fmt == O.E4M3:      # codes themselves against torch's conversion
        import torch
        with np.errstate(invalid="ignore"):
            t = torch.from_numpy((x / sc).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert np.array_equal(t[good], q[:, :77][good])


def test_oracle_gradients_against_differences():
    rng = np.random.default_rng(6)
    h, g, dy, dr = (rng.standard_normal(s) for s in ((3, 20), (20,), (3, 20), (3, 20)))
    eps, d = 1e-6, 1e-6
    loss = lambda hh, gg: (O.norm_fwd(hh, gg, eps)[0] * dy).sum() + (hh * dr).sum()
    dx, dg, _, _ = O.norm_bwd(h, g, O.norm_fwd(h, g, eps)[1], dy, dr)
    for i in ((0, 0), (1, 7), (2, 19)):
        e = np.zeros_like(h)
        e[i] = d
        assert abs((loss(h + e, g) - loss(h - e, g)) / (2 * d) - dx[i]) < 1e-7
    for i in (0, 11):
        e = np.zeros_like(g)
        e[i] = d
        assert abs((loss(h, g + e) - loss(h, g - e)) / (2 * d) - dg[i]) < 1e-7
    x = np.linspace(-6, 6, 121)
    assert np.abs((O.gelu(x + d) - O.gelu(x - d)) / (2 * d) - O.gelu_slope(x)).max() < 1e-8


def test_c_refusals():
    """Host-side checks: nothing is launched, so no device is needed (addresses are never followed)."""
    L = _lib()
    c, bad, uns, ws = L._lib, L.ERR_INVALID_ARG, L.ERR_UNSUPPORTED, L.ERR_WORKSPACE
    p, odd, one = 4096, 4096 + 2, 4096 + 1
    assert c.snack_ckpt_pack(p, 4, 32, L.F32, p, p, None) == bad           # not a checkpoint format
    assert c.snack_ckpt_pack(p, 4, 0, L.INT8, p, p, None) == bad
    assert c.snack_ckpt_pack(p, -1, 8, L.INT8, p, p, None) == bad
    assert c.snack_ckpt_pack(None, 4, 32, L.INT8, p, p, None) == bad
    assert c.snack_ckpt_pack(p, 4, 32, L.INT8, p + 8, p, None) == bad      # codes not 16-byte aligned
    assert c.snack_ckpt_pack(odd, 4, 32, L.INT8, p, p, None) == bad
    assert c.snack_ckpt_pack(p, 1 << 31, 32, L.INT8, p, p, None) == uns
    assert c.snack_ckpt_pack(p, 1 << 26, 1024, L.INT8, p, p, None) == uns  # 2^31 blocks
    assert c.snack_ckpt_pack(None, 0, 32, L.INT8, None, None, None) == L.OK
    assert c.snack_ckpt_unpack(p, p, 4, 32, L.INT8, p, L.INT8, None) == bad
    assert c.snack_ckpt_unpack(p, None, 4, 32, L.INT8, p, L.F32, None) == bad
    assert c.snack_ckpt_unpack(p, p, 4, 32, L.INT8, one, L.BF16, None) == bad
    f = ctypes.c_float
    fwd = lambda X=p, R=p, hf=L.F32, g=p, eps=1e-6, rows=4, n=32, H=p, Y=p, r=p, qf=L.F32, Q=None, S=None: \
        c.snack_rmsnorm_fwd(X, R, hf, g, f(eps), rows, n, H, Y, r, qf, Q, S, None)
    assert fwd(hf=L.INT8) == bad and fwd(eps=-1.0) == bad and fwd(eps=float("nan")) == bad
    assert fwd(R=None) == bad and fwd(H=None) == bad and fwd(r=None) == bad and fwd(g=None) == bad
    assert fwd(Y=None) == bad and fwd(Q=p) == bad and fwd(Q=p, S=p, qf=L.BF16) == bad
    assert fwd(Q=p + 8, S=p, qf=L.INT8) == bad and fwd(H=odd) == bad and fwd(hf=L.BF16, H=one) == bad
    assert fwd(rows=0, X=None) == L.OK and fwd(n=1 << 31) == uns
    need = ctypes.c_int64()
    assert c.snack_rmsnorm_bwd_work(4, 32, ctypes.byref(need)) == L.OK and need.value > 0
    assert c.snack_rmsnorm_bwd_work(4, 0, ctypes.byref(need)) == bad
    assert c.snack_rmsnorm_bwd_work(4, 32, None) == bad
    bwd = lambda H=p, HS=None, hf=L.F32, dX=p, dg=p, w=p, wb=1 << 20, rows=4, n=32: \
        c.snack_rmsnorm_bwd(H, HS, hf, p, p, p, None, rows, n, dX, dg, w, wb, None)
    assert bwd(hf=L.INT8) == bad and bwd(hf=7) == bad and bwd(dX=None) == bad and bwd(H=None) == bad
    assert bwd(w=None) == bad and bwd(wb=8) == ws and bwd(n=1 << 31) == uns
    assert bwd(dg=None, w=None, n=20000) == bad              # long rows need the scratch in any case
    assert bwd(rows=0, dg=None, H=None) == L.OK
    assert c.snack_gelu_ckpt_fwd(p, 4, 32, L.INT8, None, None, None, None, None, None) == bad
    assert c.snack_gelu_ckpt_fwd(p, 4, 32, L.INT8, p, p, None, None, None, None) == bad
    assert c.snack_gelu_ckpt_fwd(p, 4, 32, L.BF16, p, None, None, None, None, None) == bad
    assert c.snack_gelu_ckpt_bwd(p, None, p, 4, 32, L.INT8, p, None) == bad
    assert c.snack_gelu_ckpt_bwd(p, p, p, 4, 32, L.INT8, None, None) == bad
    assert c.snack_backward_ckpt(None, p, p, L.INT8, p, p, p, 4, None) == bad


def test_python_refusals():
    import torch
    L = _lib()
    x = torch.zeros(4, 40)
    for call in (lambda: L.Ckpt.pack(x, L.INT8), lambda: L.rmsnorm_fwd(x, torch.ones(40), 1e-6),
                 lambda: L.gelu_ckpt_fwd(x, L.E4M3)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(TypeError):
        L.Ckpt.pack(x.double(), L.INT8)
    with pytest.raises(ValueError):
        L.Ckpt.pack(x[0], L.INT8)
    with pytest.raises(ValueError):
        L.Ckpt(x, x, L.BF16, 40)
    with pytest.raises(TypeError):
        L.Ckpt(x, x, L.INT8, 40)
    with pytest.raises(ValueError):
        L.Ckpt(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 3, dtype=torch.uint8), L.INT8, 40)
