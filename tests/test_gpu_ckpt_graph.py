"""Layer gradients from a checkpoint recorded into a HIP graph: a replay takes the layer as it then is, and recording
leaves nothing that an eager call takes for made."""
import pytest

from snack_inputs import normal, random_layer
from tests import ckpt_oracle as O
from tests.gpu_util import assert_close, dev, host, lib, say

pytestmark = pytest.mark.gpu

# streamed passes; slice-tiled ones with several slices at 64 and at 8 columns, and the same layer at several batch
# tiles; short keys; dW by the tile list (every one of them dense enough but the short keys)
CASES = [(300, 260, 12000, 1), (300, 260, 12000, 3), (1300, 1300, 84500, 64), (4000, 4000, 800000, 8),
         (1300, 1300, 84500, 130), (3000, 900, 35003, 130), (300, 260, 700, 5)]


def _layer(M, K, nnz, B, key):
    rows, cols, vals = random_layer(M, K, nnz, key)
    return lib().SnackLayer(M, K, dev(rows), dev(cols), dev(vals), seed=6, max_batch=B)


def _against_oracle(layer, ck, dY, dX, dW):
    import numpy as np
    import oracle
    r, c, v = (host(t) for t in layer.export())
    xv = O.unpack(host(ck.q), host(ck.s), ck.fmt, ck.n).astype(np.float32)
    assert_close("dX", host(dX), *oracle.backward_dx(layer.M, layer.K, r, c, v, host(dY)))
    assert_close("dW", host(dW), *oracle.backward_dw(layer.M, layer.K, r, c, xv, host(dY)))


@pytest.mark.parametrize("stepped", [False, True])
@pytest.mark.parametrize("M,K,nnz,B", CASES)
def test_replays_follow_the_layer(M, K, nnz, B, stepped):
    """Captured as the layer's first call, its value copy fresh or stepped past; then values and positions change."""
    import torch
    L = lib()
    key = f"ckptgraph/{M}x{K}/{nnz}/{B}"
    layer = _layer(M, K, nnz, B, key)
    try:
        ck, dY = L.Ckpt.pack(dev(normal((B, K), key + "/x")), L.INT8), dev(normal((B, M), key + "/dy"))
        step = dev(normal((nnz,), key + "/step"))
        if stepped:
            layer.sgd_step(step, 0.1)
        dX, dW = torch.zeros(B, K, device="cuda"), torch.zeros(nnz, device="cuda")
        torch.cuda.synchronize()
        say("capture", key, stepped)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.backward_ckpt(ck, dY, dX=dX, dW=dW)
        say("eager before the first replay")
        _against_oracle(layer, ck, dY, *layer.backward_ckpt(ck, dY))
        changes = [lambda: layer.sgd_step(step, 0.1), lambda: layer.prune_regrow(nnz // 4),
                   lambda: layer.sgd_step(step, -0.2), lambda: layer.prune_regrow_rows(1, 4), lambda: None]
        for i, change in enumerate(changes):
            change()
            dX.zero_()
            dW.zero_()
            say("replay", i)
            g.replay()
            torch.cuda.synchronize()
            _against_oracle(layer, ck, dY, dX, dW)
            eager = layer.backward_ckpt(ck, dY)
            assert torch.equal(dX, eager[0]) and torch.equal(dW, eager[1])
    finally:
        layer.close()


@pytest.mark.parametrize("M,K,nnz,B", CASES[1:5])
def test_captured_step_and_eager_calls(M, K, nnz, B):
    """Gradients and SGD step in one graph, eager gradients between its replays: the bits of a layer stepped eagerly."""
    import torch
    L = lib()
    key = f"ckptgraph/step/{M}x{K}/{nnz}/{B}"
    layer, twin = _layer(M, K, nnz, B, key), _layer(M, K, nnz, B, key)
    try:
        ck, dY = L.Ckpt.pack(dev(normal((B, K), key + "/x")), L.E4M3), dev(normal((B, M), key + "/dy"))
        dX, dW = torch.zeros(B, K, device="cuda"), torch.zeros(nnz, device="cuda")
        torch.cuda.synchronize()
        say("capture step", key)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.backward_ckpt(ck, dY, dX=dX, dW=dW)
            layer.sgd_step(dW, 0.05)
        for i in range(4):
            say("replay", i)
            g.replay()
            torch.cuda.synchronize()
            tX, tW = twin.backward_ckpt(ck, dY)
            assert torch.equal(dX, tX) and torch.equal(dW, tW)
            twin.sgd_step(tW, 0.05)
            a, b = layer.backward_ckpt(ck, dY), twin.backward_ckpt(ck, dY)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    finally:
        layer.close()
        twin.close()


@pytest.mark.parametrize("want_dx", [True, False])
@pytest.mark.parametrize("M,K,nnz,B", CASES)
def test_captured_fused_step(M, K, nnz, B, want_dx):
    """The gradients with the step in one call: every replay as an eagerly stepped layer, eager calls between them."""
    import torch
    key = f"ckptgraph/fused/{M}x{K}/{nnz}/{B}"
    layer, twin = _layer(M, K, nnz, B, key), _layer(M, K, nnz, B, key)
    try:
        X, dY = dev(normal((B, K), key + "/x")), dev(normal((B, M), key + "/dy"))
        dX, dW = torch.zeros(B, K, device="cuda"), torch.zeros(nnz, device="cuda")
        torch.cuda.synchronize()
        say("capture fused", key, want_dx)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.backward_sgd(X, dY, 0.05, want_dx=want_dx, dX=dX, dW=dW)
        for i in range(4):
            say("replay", i)
            g.replay()
            torch.cuda.synchronize()
            tX, tW = twin.backward_sgd(X, dY, 0.05, want_dx=want_dx)
            assert torch.equal(dW, tW) and (not want_dx or torch.equal(dX, tX))
            if i:      # the first two replays with nothing between them
                assert torch.equal(layer.backward(X, dY)[0], twin.backward(X, dY)[0])
    finally:
        layer.close()
        twin.close()


def test_bf16_copy_is_made_where_it_is_read():
    """The inference forward's 16-bit values: recording the call that makes them makes none, and a step replayed from
    a graph moves the values past them."""
    import numpy as np
    import torch
    L = lib()
    M, K, nnz, key = 300, 260, 12000, "ckptgraph/bf16"
    layer, twin = _layer(M, K, nnz, 2, key), _layer(M, K, nnz, 2, key)
    try:
        X, step = dev(normal((2, K), key + "/x")), dev(normal((nnz,), key + "/step"))
        Y, E, T = (torch.zeros(2, M, device="cuda") for _ in range(3))
        torch.cuda.synchronize()
        say("bf16 capture")
        g, gs = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            L.snack_forward_infer(layer.h, X, Y, bf16_values=True)
        L.snack_forward_infer(layer.h, X, E, bf16_values=True)      # before the first replay
        L.snack_forward_infer(twin.h, X, T, bf16_values=True)
        assert torch.equal(E, T) and np.abs(host(T)).max() > 0
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, T)
        with torch.cuda.graph(gs):
            layer.sgd_step(step, 0.5)
        for i in range(3):
            say("bf16 replay", i)
            gs.replay()
            torch.cuda.synchronize()
            twin.sgd_step(step, 0.5)
            L.snack_forward_infer(layer.h, X, E, bf16_values=True)
            L.snack_forward_infer(twin.h, X, T, bf16_values=True)
            assert torch.equal(E, T)
    finally:
        layer.close()
        twin.close()
