"""Input gradients of wide and of very large calls against bounds that do not
grow with the width (sparse_gradient.py): every width class of the activation's
backward pass, on both sides of its edges and past the last."""
import numpy as np
import pytest
import torch

import fused_ref as ref
import sparse_gradient as sparse
from quantized_linear_layers_token_b200 import synth
from test_gpu_fused import Layer, cuda, host, q, within  # noqa: F401 (q: fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [1040, 4112, 8208, 12304, 16400, 24592, 32768, 32784, 40000])
@pytest.mark.parametrize("gated", [False, True])
def test_wide_layers(q, oracle, gated, N):  # noqa: F811
    for M, act, with_dbias in ((3, "silu", True), (310, "gelu_tanh", True), (5, "gelu", False), (40, "relu", False)):
        L = Layer(q, oracle, synth.W8_PERCHANNEL, M, 128, N, 2, gated=gated)
        rng = np.random.default_rng([M, N])
        Z = (rng.standard_normal((M, N)) * 1.5).astype(np.float16)
        dY, at = sparse.gradient(M, N, gated, rng)
        dX = torch.full((M, 128), float("nan"), dtype=torch.float16, device="cuda")
        db = torch.full((N,), float("nan"), device="cuda") if with_dbias else None
        n = (q.qlin_backward_gated_workspace if gated else q.qlin_backward_act_workspace)(M, L.w)
        (q.qlin_backward_gated if gated else q.qlin_backward_act)(L.w, cuda(dY), cuda(Z), M, cuda(L.s), dX, db,
                                                                    q.empty_workspace(n), n, act=ref.ACTS.index(act))
        q.qlin_poll_device_status()
        _, want, bound = sparse.reference(act, gated, dY, Z, at, L.pk, L.W, L.s)
        within(host(dX), want, bound, (M, "dX"))
        if with_dbias:
            assert np.all(np.delete(host(db), at) == 0)


@pytest.mark.parametrize("gated", [False, True])
def test_buffers_past_31_bits(q, oracle, gated):  # noqa: F811
    """The last rows of a call whose dZ passes 2^31 elements against 64 bits."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    M, K, N, last = 68003, 256, 32768, 300
    gen = torch.Generator(device="cuda").manual_seed(5)
    W = (torch.randn(K, N, generator=gen, device="cuda") * 0.05).half()
    layer = q.PackedLayer.pack(W, np.zeros(0, np.int32), synth.W8_PERCHANNEL)
    rng = np.random.default_rng(1)
    d, at = sparse.gradient(last, N, gated, rng)
    dY = torch.zeros(M, d.shape[1], dtype=torch.float16, device="cuda")
    dY[-last:] = cuda(d)
    Z = torch.empty(M, N, dtype=torch.float16, device="cuda").normal_(generator=gen)
    dX = torch.empty(M, K, dtype=torch.float16, device="cuda")
    n = (q.qlin_backward_gated_workspace if gated else q.qlin_backward_act_workspace)(M, layer.w)
    (q.qlin_backward_gated if gated else q.qlin_backward_act)(layer.w, dY, Z, M, None, dX, None, q.empty_workspace(n), n,
                                                                act=4)
    q.qlin_poll_device_status()
    assert (dX[:-last] == 0).all()
    pk = oracle.pack_layer(host(W).view(np.uint16), np.zeros(0, np.int32), synth.W8_PERCHANNEL)
    _, want, bound = sparse.reference("silu", gated, d, host(Z[-last:]), at, pk, host(W), np.zeros(0, np.float32))
    within(host(dX[-last:]), want, bound, "dX")
    del dX, dY, Z
    torch.cuda.empty_cache()
