"""The sharp checks of wide layers are sharp: a lost last vector, a lost last
step and an error of one percent each exceed the bound (no GPU needed)."""
import numpy as np
import pytest

import fused_ref as ref
import sparse_gradient as sparse
from quantized_linear_layers_token_b200 import synth


@pytest.mark.parametrize("N", [1040, 16400, 32784, 40000])
@pytest.mark.parametrize("gated", [False, True])
def test_bound_catches_losses(oracle, gated, N):
    M, K, nO = 5, 128, 2
    rng = np.random.default_rng([N, gated])
    O = np.sort(rng.choice(K, nO, replace=False)).astype(np.int32)
    W = (rng.standard_normal((K, N)) * 0.02).astype(np.float16)
    pk = oracle.pack_layer(W.view(np.uint16), O, synth.W8_PERCHANNEL)
    s = rng.uniform(1, 8, nO).astype(np.float32)
    Z = (rng.standard_normal((M, N)) * 1.5).astype(np.float16)
    dY, at = sparse.gradient(M, N, gated, rng)
    dz, want, bound = sparse.reference("silu", gated, dY, Z, at, pk, W, s)

    def dx(d):
        z = np.zeros((M, len(at)))
        part = {"B": pk["B"][:, at], "cscale": pk["cscale"][at], "O": O}
        return ref.input_gradient(d, z, np.ones(M), part, W[:, at], s)[0]

    assert np.array_equal(dx(dz), want)
    for lost in (at >= N - 8, at >= (N - 1) // 64 * 64, at < 8):
        d = dz.copy()
        d[:, lost] = 0
        assert (np.abs(dx(d) - want) / bound).max() > 4
    assert (np.abs(dx(1.01 * dz) - want) / bound).max() > 1
