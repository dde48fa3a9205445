"""The operators together, as a training step uses them: the example's block against the same formulas in 64 bits."""
import importlib.util
import math
import os

import pytest

from tests.gpu_util import lib, say

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "checkpointed_block.py")
    spec = importlib.util.spec_from_file_location("checkpointed_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _dense(layer):
    import torch
    r, c, v = layer.export()
    w = torch.zeros(layer.M, layer.K, dtype=torch.float64)
    w[r.cpu().long(), c.cpu().long()] = v.cpu().double()
    return w, r.cpu().long(), c.cpu().long()


@pytest.mark.parametrize("fmt", ["INT8", "E4M3"])
@pytest.mark.parametrize("rows,width,hidden,sparsity", [(3, 70, 130, 80), (65, 100, 300, 95), (130, 96, 257, 60)])
def test_block_gradients(rows, width, hidden, sparsity, fmt):
    """The step's gradients against 64-bit products of the values that were kept."""
    import torch
    L, ex = lib(), _example()
    say("block", rows, width, hidden, fmt)
    block = ex.CheckpointedBlock(width, hidden, sparsity, rows, getattr(L, fmt))
    try:
        g = torch.Generator().manual_seed(3)
        res, x = torch.randn(rows, width, generator=g).bfloat16(), torch.randn(rows, width, generator=g)
        d = torch.randn(rows, width, generator=g)
        block.gain += torch.randn(width, generator=g).cuda() * 0.1
        branch, h = block.forward(x.cuda(), res.cuda())
        d_x, d_gain, d_up, d_down = (t.cpu().double() for t in block.backward(d.cuda()))
        hd, rstd, ck_y, ck_a, ck_g = block.kept
        assert ck_y.fmt == ck_a.fmt == ck_g.fmt == getattr(L, fmt)
        y, a, q = (c.unpack().cpu().double() for c in (ck_y, ck_a, ck_g))
        hd, r, gain, d = hd.cpu().double(), rstd.cpu().double()[:, None], block.gain.cpu().double(), d.double()
        w_up, ru, cu = _dense(block.up)
        w_dn, rd, cd = _dense(block.down)
        # five operators of sums of at most `hidden` terms in fp32, each sum's error within its length in half
        # steps of the sum of its terms' magnitudes; the chain multiplies magnitudes, so bounds go along with it
        u = 2.0 ** -24
        n = 2 * (hidden + width + rows)
        dg, dg_m = d @ w_dn, d.abs() @ w_dn.abs()
        slope = 0.5 * torch.special.erfc(-a / math.sqrt(2)) + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)
        da, da_m = dg * slope, dg_m * 1.13                  # |slope| <= 1.13
        dy, dy_m = da @ w_up, da_m @ w_up.abs()
        xh, w, w_m = hd * r, dy * gain, dy_m * gain.abs()
        want = r * (w - xh * (w * xh).mean(-1, keepdim=True)) + d
        mag = r * (w_m + xh.abs() * (w_m * xh.abs()).mean(-1, keepdim=True)) + d.abs()
        assert (d_x - want).abs().le(n * u * mag).all()
        assert (d_gain - (dy * xh).sum(0)).abs().le(n * u * (dy_m * xh.abs()).sum(0)).all()
        assert (d_down - (d.t() @ q)[rd, cd]).abs().le(n * u * (d.abs().t() @ q.abs())[rd, cd]).all()
        assert (d_up - (da.t() @ y)[ru, cu]).abs().le(n * u * (da_m.t() @ y.abs())[ru, cu]).all()
        blocks = lambda k: -(-k // 32)
        assert block.kept_bytes() == rows * (2 * width + 4 + 33 * (blocks(width) + 2 * blocks(hidden)))
    finally:
        block.close()


def test_block_step_lowers_the_loss():
    """A small step lr along the gradient g lowers the loss by lr |g|^2, to the curvature (0.4 % of it at lr = 0.1 for
    blocks of this size in 64 bits) and the checkpoints' rounding (half a step in 127 or more of a block's largest
    value, under 1 % of g); then 60 steps with drop/regrow between them."""
    import torch
    ex = _example()
    say("block step")
    block = ex.CheckpointedBlock(96, 384, 90, 64)
    try:
        g = torch.Generator(device="cuda").manual_seed(4)
        res = torch.randn(64, 96, device="cuda", generator=g).bfloat16()
        x, target = (torch.randn(64, 96, device="cuda", generator=g) for _ in range(2))
        branch, h = block.forward(x, res)
        err = branch + h.float() - target
        grads = block.backward(err * (2.0 / err.numel()))[1:]
        n2 = sum(float((v.double() ** 2).sum()) for v in grads)
        before = float(block.step(x, res, target, 0.1))
        losses = [float(block.step(x, res, target, 1.0))]
        assert abs((before - losses[0]) / (0.1 * n2) - 1) < 0.05
        for i in range(60):
            losses.append(float(block.step(x, res, target, 1.0)))
            if i % 20 == 19:
                block.up.prune_regrow(block.up.nnz // 50)
        assert all(math.isfinite(v) for v in losses) and losses[-1] < 0.75 * losses[0], losses
    finally:
        block.close()
