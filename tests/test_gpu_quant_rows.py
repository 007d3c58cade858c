"""The quantization kernel at many rows, where its row takes fewer threads:
codes and scales are the oracle's, bit for bit."""
import numpy as np
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


@pytest.mark.parametrize("update", [False, True])
@pytest.mark.parametrize("M,K,nO", [(1300, 32, 3), (700, 1024, 0), (700, 992, 130), (1300, 1056, 11), (1201, 4096, 41),
                                    (1300, 4128, 300), (1250, 8192, 1), (1300, 8224, 7), (1190, 16384, 600)])
def test_many_rows(q, oracle, M, K, nO, update):
    rng = np.random.default_rng([M, K, nO])
    X = rng.standard_normal((M, K)).astype(np.float16)
    O = np.sort(rng.choice(K, nO, replace=False)).astype(np.int32)
    X[:, O] *= 12
    X[5] = 0
    X[M - 1] *= 1000
    W = (rng.standard_normal((K, 16)) * 0.05).astype(np.float16)
    layer = q.PackedLayer.pack(torch.from_numpy(W).cuda(), O, synth.W8_PERCHANNEL)
    s0 = (1 + rng.random(nO)).astype(np.float32)
    s = torch.from_numpy(s0).cuda()
    Xq = torch.full((M + 1, K), 77, dtype=torch.int8, device="cuda")
    XqO = torch.full((M + 1, nO), 77, dtype=torch.int8, device="cuda")
    a = torch.full((M + 1,), 77.0, device="cuda")
    n = q.qlin_quant_act_workspace(M, layer.w)
    q.qlin_quant_act(torch.from_numpy(X).cuda(), M, layer.w, s, 0.9, update, Xq, a, XqO, q.empty_workspace(n), n)
    q.qlin_poll_device_status()
    pk = oracle.pack_layer(W.view(np.uint16), O, synth.W8_PERCHANNEL)
    want = oracle.momentum_update(X.view(np.uint16), O, pk["wmaxO"], 0.9, s0) if update and nO else s0
    assert np.array_equal(s.cpu().numpy().view(np.uint32), want.view(np.uint32))
    wq, wa, wo = oracle.quant_act(X.view(np.uint16), O, want)
    assert np.array_equal(Xq[:M].cpu().numpy(), wq)
    assert np.array_equal(a[:M].cpu().numpy().view(np.uint32), wa.view(np.uint32))
    if nO:
        assert np.array_equal(XqO[:M].cpu().numpy(), wo)
    # rows behind the last
    assert (Xq[M] == 77).all() and (XqO[M] == 77).all() and a[M] == 77
