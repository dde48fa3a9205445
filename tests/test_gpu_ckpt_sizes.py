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
