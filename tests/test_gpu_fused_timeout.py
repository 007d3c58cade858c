"""Device-side bounded waits of the fused layers' kernels and of their backward
pass: with a limit of zero the first wait for data that has not yet
arrived gives up, the status word says so, and the same call with the default
limit is right again.  No fault is provoked."""
import pytest
import torch

from quantized_linear_layers_token_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_linear_layers_token_b200 import qlin
    qlin.lib()
    return qlin


def run_out(q, call, outputs, zero=()):
    """`call` with the default limit, with none, and with the default again."""
    for t in zero:
        t.zero_()
    call()
    q.qlin_poll_device_status()
    want = [t.clone() for t in outputs]
    with q.knobs(wait_ns=0):
        call()
        with pytest.raises(q.QlinError) as e:
            q.qlin_poll_device_status()
        assert q.STATUS[e.value.status] == "QLIN_ERR_TIMEOUT"
    for t in zero:  # an aborted call may leave its workspace in any state
        t.zero_()
    for t in outputs:
        t.fill_(float("nan"))
    call()
    q.qlin_poll_device_status()
    for a, b in zip(want, outputs):
        assert torch.equal(a, b)


def layer_and_inputs(q, M, K, N, nO):
    """Long reductions, so that the wait for a tile's products cannot be over
    at its first test."""
    import numpy as np
    O = np.arange(nO, dtype=np.int32) * 11
    W = (torch.randn(K, N, device="cuda") * 0.02).half()
    layer = q.PackedLayer.pack(W, O, synth.W8_PERCHANNEL)
    return layer, torch.randn(M, K, device="cuda").half(), torch.full((nO,), 2.0, device="cuda")


@pytest.mark.parametrize("nO", [0, 7])
def test_fused_layers(q, nO):
    M, K, N = 600, 32768, 2048
    layer, X, s = layer_and_inputs(q, M, K, N, nO)
    n = q.qlin_forward_act_workspace(M, layer.w)
    ws = q.empty_workspace(n)
    Y, Z = torch.empty(M, N, device="cuda").half(), torch.empty(M, N, device="cuda").half()
    H, R = torch.empty(M, N // 2, device="cuda").half(), torch.randn(M, N, device="cuda").half()
    run_out(q, lambda: q.qlin_forward_act(X, M, layer.w, s, 0.9, False, Y, ws, n, act=4, residual=R), [Y], [ws])
    run_out(q, lambda: q.qlin_forward_gated(X, M, layer.w, s, 0.9, False, H, ws, n, Z=Z), [H, Z], [ws])


def test_backward(q):
    M, K, N = 2048, 1024, 32768
    layer, _, s = layer_and_inputs(q, M, K, N, 7)
    dH, Z = torch.randn(M, N // 2, device="cuda").half(), torch.randn(M, N, device="cuda").half()
    n = q.qlin_backward_gated_workspace(M, layer.w)
    ws = q.empty_workspace(n)
    dX, db = torch.empty(M, K, device="cuda").half(), torch.empty(N, device="cuda")
    run_out(q, lambda: q.qlin_backward_gated(layer.w, dH, Z, M, s, dX, db, ws, n), [dX, db])
