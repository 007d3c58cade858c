"""Buffers past 2^31 elements: the last rows of a large call are those of a
call on these rows alone."""
import numpy as np
import pytest
import torch

from quantized_linear_layers_token_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    from quantized_linear_layers_token_b200 import qlin
    qlin.lib()
    yield qlin
    torch.cuda.empty_cache()


def half(*shape):
    return torch.randn(*shape, device="cuda", dtype=torch.float16)


@pytest.mark.parametrize("rms", [False, True])
def test_norms(q, rms):
    M, K, last = 270001, 8192, 37
    kind = q.QLIN_NORM_RMS if rms else q.QLIN_NORM_LAYER
    X, dY = half(M, K), half(M, K)
    gamma = torch.rand(K, device="cuda") + 0.5

    def run(X, dY):
        M = X.shape[0]
        Y, dX = torch.empty_like(X), torch.empty_like(X)
        mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        dg = torch.empty(K, device="cuda")
        n = q.qlin_norm_backward_workspace(M, K)
        q.qlin_norm_forward(X, M, K, kind, gamma, None, 1e-5, Y, None if rms else mean, rstd)
        q.qlin_norm_backward(dY, X, M, K, kind, gamma, None if rms else mean, rstd, dY, dX, dg, None,
                             q.empty_workspace(n), n)
        q.qlin_poll_device_status()
        return Y, rstd, dX, dg

    Y, rstd, dX, dg = run(X, dY)
    y, r, dx, _ = run(X[-last:].clone(), dY[-last:].clone())
    # the statistics' sums may be split over another number of threads: a few
    # fp32 roundings (relative 2^-24 each, 14 levels), then one of fp16 each
    assert ((rstd[-last:] - r).abs() <= 2.0 ** -19 * r).all()
    for a, b in ((Y[-last:], y), (dX[-last:], dx)):
        a, b = a.double(), b.double()
        assert ((a - b).abs() <= 2.0 ** -10 * b.abs() + 2.0 ** -15).all()
    # dgamma of standard normal rows: a sum of M terms of unit variance, 8 of its deviations
    assert dg.abs().max() < 8 * M ** 0.5


@pytest.mark.parametrize("gated", [False, True])
def test_fused_layers(q, gated):
    M, K, N, last = 68003, 256, 32768, 300
    O = np.zeros(0, dtype=np.int32)
    W = half(K, N) * 0.05
    layer = q.PackedLayer.pack(W, O, synth.W8_PERCHANNEL)
    X, s = half(M, K), torch.empty(0, device="cuda")
    dY = half(M, N // 2 if gated else N)

    def run(X, dY):
        M = X.shape[0]
        Y, Z = torch.empty_like(dY), torch.empty(M, N, device="cuda", dtype=torch.float16)
        dX, db = torch.empty_like(X), torch.empty(N, device="cuda")
        n = (q.qlin_forward_gated_workspace if gated else q.qlin_forward_act_workspace)(M, layer.w)
        (q.qlin_forward_gated if gated else q.qlin_forward_act)(X, M, layer.w, s, 0.9, False, Y, q.empty_workspace(n), n,
                                                                act=4, Z=Z)
        n = (q.qlin_backward_gated_workspace if gated else q.qlin_backward_act_workspace)(M, layer.w)
        back = q.qlin_backward_gated if gated else q.qlin_backward_act
        back(layer.w, dY, Z, M, s, dX, db, q.empty_workspace(n), n, act=4)
        q.qlin_poll_device_status()
        return Y, Z, dX

    Y, Z, dX = run(X, dY)
    y, z, dx = run(X[-last:].clone(), dY[-last:].clone())
    # exact sums, then the same fp32 operations: the same bits
    assert torch.equal(Y[-last:], y) and torch.equal(Z[-last:], z)
    # dX: the same fp16 products, N of them added in fp32 in another order
    # (relative to the sum of magnitudes, at most 2 N 2^-24), one fp16 rounding
    # on either side (2^-11 each).  |dZ| <= 1.1 |dY| (slope), gated 1.1 |dY| |up| or |dY| |act| <= |dY| |z|
    zz, g = z.double().abs(), dy_abs(dY[-last:], gated)
    d = g * 1.1 * (torch.stack((zz[:, 1::2], zz[:, 0::2]), 2).flatten(1) if gated else 1.0)
    mag = d @ (W.double().abs().t() * 1.01 + 0.001)
    assert ((dX[-last:].double() - dx.double()).abs() <= 2 * N * 2.0 ** -24 * mag + 2.0 ** -10 * dx.double().abs() + 2.0 ** -24).all()


def dy_abs(dY, gated):
    a = dY.double().abs()
    return a.repeat_interleave(2, 1) if gated else a
