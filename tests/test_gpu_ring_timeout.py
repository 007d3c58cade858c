"""The row rings of the norms and of the activation's backward pass with waits
that have no time: a call whose waits run out ends in the time of its rows (a
thread gives up once, not once a row) and says so, one whose data was there in
time is right, and the same call with the default limit is right again.  No
fault is provoked."""
import time

import pytest
import torch

from quantized_linear_layers_token_b200 import synth
from test_gpu_ffn import q  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def check(q, call, outputs):  # noqa: F811
    call()
    q.qlin_poll_device_status()
    want = [t.clone() for t in outputs]
    for _ in range(5):
        gave_up = False
        with q.knobs(wait_ns=0):
            t0 = time.perf_counter()
            call()
            try:
                q.qlin_poll_device_status()
            except q.QlinError as e:
                assert q.STATUS[e.status] == "QLIN_ERR_TIMEOUT"
                gave_up = True
            assert time.perf_counter() - t0 < 4
        assert gave_up or all(torch.equal(a, b) for a, b in zip(outputs, want))
    for t in outputs:
        t.fill_(float("nan"))
    call()
    q.qlin_poll_device_status()
    assert all(torch.equal(a, b) for a, b in zip(outputs, want))


@pytest.mark.parametrize("K", [64, 512, 4096, 16384])
def test_norms(q, K):  # noqa: F811
    M = (1 << 28) // K
    X, dY = torch.randn(M, K, device="cuda").half(), torch.randn(M, K, device="cuda").half()
    gamma, mean, rstd = torch.rand(K, device="cuda") + 0.5, torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    Y, dX, dg = torch.empty_like(X), torch.empty_like(X), torch.empty(K, device="cuda")
    check(q, lambda: q.qlin_norm_forward(X, M, K, q.QLIN_NORM_LAYER, gamma, None, 1e-5, Y, mean, rstd), [Y, mean, rstd])
    n = q.qlin_norm_backward_workspace(M, K)
    ws = q.empty_workspace(n)
    check(q, lambda: q.qlin_norm_backward(dY, X, M, K, q.QLIN_NORM_LAYER, gamma, mean, rstd, None, dX, dg, None, ws, n),
          [dX, dg])


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("N", [528, 4096, 24576])
def test_activation(q, gated, N):  # noqa: F811
    M = (1 << 27) // N
    layer = q.PackedLayer(128, N, synth.W8_PERCHANNEL, 0)
    dY = torch.randn(M, N // 2 if gated else N, device="cuda").half()
    Z, db = torch.randn(M, N, device="cuda").half(), torch.empty(N, device="cuda")
    n = q.qlin_backward_act_workspace(M, layer.w)
    ws = q.empty_workspace(n)
    back = q.qlin_backward_gated if gated else q.qlin_backward_act
    check(q, lambda: back(layer.w, dY, Z, M, None, None, db, ws, n, act=4), [db])
