"""Bounded waits of the fused layer on CTA pairs that run out while a pair
still has tiles to come: the residual's loads stop, what is on its way lands,
and the same call with the default limit is right again.  No fault is
provoked."""
import pytest
import torch

from quantized_linear_layers_token_b200 import synth
from test_gpu_fused_timeout import layer_and_inputs, q, run_out  # noqa: F401 (q: fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("keep_z", [False, True])
@pytest.mark.parametrize("nO", [0, 7])
def test_residual_with_several_tiles_per_pair(q, nO, keep_z):  # noqa: F811
    M, K, N = 2560, 16384, 6144  # 240 tiles on at most 74 pairs
    layer, X, s = layer_and_inputs(q, M, K, N, nO)
    assert layer.fmt == synth.W8_PERCHANNEL
    n = q.qlin_forward_act_workspace(M, layer.w)
    ws = q.empty_workspace(n)
    R = torch.randn(M, N, device="cuda").half()
    Y = torch.empty_like(R)
    Z = torch.empty_like(R) if keep_z else None
    run_out(q, lambda: q.qlin_forward_act(X, M, layer.w, s, 0.9, False, Y, ws, n, act=4, residual=R, Z=Z),
            [Y, Z] if keep_z else [Y], [ws])
