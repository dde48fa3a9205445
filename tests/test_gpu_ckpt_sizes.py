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
