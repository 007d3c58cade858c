"""Host-side checks of the fused layers, the gated block and the norms (no GPU
needed): refusals before anything is enqueued, and the references' gradients
against differences."""
import numpy as np
import pytest

import fused_ref as ref


@pytest.fixture(scope="module")
def q():
    from quantized_linear_layers_token_b200 import build, qlin
    build.build()
    return qlin


A, B, C, D, E, F, G = (1 << n for n in range(24, 31))  # addresses that are never touched


def status(q, call, *args, **kw):
    with pytest.raises(q.QlinError) as e:
        call(*args, stream=0, **kw)
    return q.STATUS[e.value.status][9:]


def weights(q, K=512, N=128, fmt=0, nO=5):
    return q.qlin_weights_bind(K, N, fmt, nO, 1 << 20, q.qlin_weights_bytes(K, N, fmt, nO))


@pytest.mark.parametrize("gated", [False, True])
def test_forward_refusals(q, gated):
    w = weights(q)
    fwd = q.qlin_forward_gated if gated else q.qlin_forward_act
    n = (q.qlin_forward_gated_workspace if gated else q.qlin_forward_act_workspace)(16, w)
    assert n >= 16 * 512 + 4 * 16 + 16 * 5 + 2 * 16 * 8 * 2  # Xq, a, XqO and the compensation operand

    def call(X=A, M=16, s=B, gamma=0.9, Y=C, ws=D, size=n, **kw):
        return status(q, fwd, X, M, w, s, gamma, True, Y, ws, size, **kw)

    assert call(M=-1) == "ARG" and call(X=None) == "ARG" and call(Y=None) == "ARG" and call(s=None) == "ARG"
    assert call(gamma=1.5) == "ARG" and call(gamma=float("nan")) == "ARG"
    assert call(act=5) == "ARG" and call(act=-1) == "ARG"
    assert call(Z=C) == "ARG"  # Z and the output may not be one buffer
    assert call(size=n - 1) == "WORKSPACE" and call(ws=None) == "WORKSPACE"
    assert call(ws=D + 16) == "ALIGN"
    for kw in ({"X": A + 2}, {"Y": C + 8}, {"s": B + 4}, {"bias": E + 4}, {"Z": E + 2}):
        assert call(**kw) == "ALIGN", kw
    if not gated:
        assert call(residual=E + 2) == "ALIGN" and call(Z=E, residual=E) == "ARG"
    fwd(None, 0, w, None, 0.9, True, None, None, 0, stream=0)  # no tokens: nothing to do


@pytest.mark.parametrize("gated", [False, True])
def test_backward_refusals(q, gated):
    w = weights(q)
    bwd = q.qlin_backward_gated if gated else q.qlin_backward_act
    size = q.qlin_backward_gated_workspace if gated else q.qlin_backward_act_workspace
    n = size(16, w)
    assert size(0, w) == 0 and n >= 16 * 128 * 2

    def call(dY=A, Z=B, M=16, s=C, dX=D, dbias=None, ws=E, size=n, **kw):
        return status(q, bwd, w, dY, Z, M, s, dX, dbias, ws, size, **kw)

    assert call(M=-1) == "ARG" and call(dY=None) == "ARG" and call(s=None) == "ARG"
    assert call(dX=None) == "ARG"  # no output wanted
    assert call(Z=None, act=q.QLIN_ACT_SILU) == "ARG"
    assert call(act=9) == "ARG"
    assert call(M=65535 * 128 + 1) == "SHAPE"
    assert call(size=n - 1) == "WORKSPACE" and call(ws=None) == "WORKSPACE" and call(ws=E + 128) == "ALIGN"
    for kw in ({"dY": A + 2}, {"Z": B + 8}, {"s": C + 4}, {"dX": D + 2}, {"dbias": F + 8}):
        assert call(**kw) == "ALIGN", kw


def test_pack_gated_refusals(q):
    w = weights(q, nO=3)
    O = np.array([1, 2, 3], np.int32)
    assert status(q, q.qlin_pack_gated, None, B, O, w) == "ARG"
    assert status(q, q.qlin_pack_gated, A, B + 8, O, w) == "ALIGN"
    for bad in ([3, 2, 1], [1, 1, 2], [1, 2, 512]):
        assert status(q, q.qlin_pack_gated, A, B, np.array(bad, np.int32), w) == "ARG"


def test_norm_refusals(q):
    def fwd(X=A, M=4, K=64, kind=0, gamma=B, beta=None, eps=1e-5, Y=C, **kw):
        return status(q, q.qlin_norm_forward, X, M, K, kind, gamma, beta, eps, Y, **kw)

    assert fwd(M=-1) == "ARG" and fwd(K=0) == "ARG" and fwd(kind=2) == "ARG" and fwd(kind=-1) == "ARG"
    assert fwd(K=48) == "SHAPE" and fwd(K=65568) == "SHAPE"
    for eps in (0.0, -1e-5, float("nan"), float("inf")):
        assert fwd(eps=eps) == "ARG"
    assert fwd(X=None) == "ARG" and fwd(gamma=None) == "ARG" and fwd(Y=None) == "ARG"
    for kw in ({"X": A + 2}, {"gamma": B + 4}, {"beta": B + 4}, {"Y": C + 2}, {"mean": D + 4}, {"rstd": D + 4}):
        assert fwd(**kw) == "ALIGN", kw
    n = q.qlin_norm_backward_workspace(4, 64)

    def bwd(dY=A, X=B, M=4, K=64, kind=0, gamma=C, mean=D, rstd=E, dres=None, dX=F, dgamma=G, dbeta=None, ws=1 << 31,
            size=n):
        return status(q, q.qlin_norm_backward, dY, X, M, K, kind, gamma, mean, rstd, dres, dX, dgamma, dbeta, ws, size)

    assert bwd(M=-1) == "ARG" and bwd(K=40) == "SHAPE" and bwd(kind=7) == "ARG"
    assert bwd(dX=None, dgamma=None) == "ARG" and bwd(mean=None) == "ARG" and bwd(rstd=None) == "ARG"
    assert bwd(dY=None) == "ARG" and bwd(X=None) == "ARG" and bwd(gamma=None) == "ARG"
    assert bwd(size=n - 1) == "WORKSPACE" and bwd(ws=None) == "WORKSPACE" and bwd(ws=(1 << 31) + 16) == "ALIGN"
    for kw in ({"dY": A + 2}, {"X": B + 2}, {"gamma": C + 4}, {"mean": D + 4}, {"rstd": E + 4}, {"dres": A + 2},
               {"dX": F + 2}, {"dgamma": G + 4}, {"dbeta": G + 4}):
        assert bwd(**kw) == "ALIGN", kw
    with pytest.raises(q.QlinError):
        q.qlin_norm_backward_workspace(-1, 64)


def test_binding_refuses_host_tensors(q):
    import torch
    w = weights(q, nO=0)
    x = torch.zeros(16, 512, dtype=torch.float16)
    with pytest.raises(ValueError):
        q.qlin_forward_act(x, 16, w, None, 0.9, False, C, D, 1 << 20, stream=0)
    with pytest.raises(ValueError):
        q.qlin_norm_forward(x.float(), 16, 512, 0, B, None, 1e-5, C, stream=0)
    with pytest.raises(ValueError):
        q.PackedLayer.pack_gated(x, x[:8], np.zeros(0, np.int32), 0)


# ---------------------------------------------------------------- the references

@pytest.mark.parametrize("name", ref.ACTS)
def test_slopes_against_differences(name):
    z = np.linspace(-8, 8, 1601) + 0.003
    h = 1e-5
    num = (ref.act(name, z + h)[0] - ref.act(name, z - h)[0]) / (2 * h)
    assert np.max(np.abs(num - ref.act(name, z)[1])) < 1e-8
    assert np.max(np.abs(ref.act(name, z)[1])) < 1.13  # the kernels' row scale counts on it


def test_reference_gradients_against_differences():
    """dX, dbias, dgamma, dbeta of the references against central differences
    of the forward formulas in 64 bits."""
    rng = np.random.default_rng(3)
    x, gamma, beta = rng.standard_normal((4, 32)), rng.standard_normal(32), rng.standard_normal(32)
    dy, dres = rng.standard_normal((4, 32)), np.zeros((4, 32))
    h = 1e-6
    for rms in (False, True):
        def loss(x, g, b):
            return float((ref.norm_forward(x, g, b, 1e-5, rms)[0] * dy).sum())
        _, _, mu, r, _, _ = ref.norm_forward(x, gamma, beta, 1e-5, rms)
        dx, _, dg, _, db, _ = ref.norm_backward(dy, x, gamma, mu, r, dres, rms)
        for i, k in [(0, 0), (3, 31), (2, 7)]:
            e = np.zeros_like(x)
            e[i, k] = h
            assert abs((loss(x + e, gamma, beta) - loss(x - e, gamma, beta)) / (2 * h) - dx[i, k]) < 1e-6
        e = np.zeros(32)
        e[5] = h
        assert abs((loss(x, gamma + e, beta) - loss(x, gamma - e, beta)) / (2 * h) - dg[5]) < 1e-6
        assert abs((loss(x, gamma, beta + e) - loss(x, gamma, beta - e)) / (2 * h) - db[5]) < 1e-6
    # the gated product, through a linear map z = x We + b
    We, b = rng.standard_normal((32, 12)), rng.standard_normal(12)
    dh = rng.standard_normal((4, 6))
    zero = np.zeros((4, 12))
    for name in ref.ACTS:
        def gated(x, b):
            return float((ref.forward_gated(x @ We + b, zero, name)[0] * dh).sum())
        dz, _ = ref.dz_gated(dh, x @ We + b, name)
        e = np.zeros_like(x)
        e[1, 9] = h
        assert abs((gated(x + e, b) - gated(x - e, b)) / (2 * h) - (dz @ We.T)[1, 9]) < 1e-5
        e = np.zeros(12)
        e[4] = h
        assert abs((gated(x, b + e) - gated(x, b - e)) / (2 * h) - dz.sum(0)[4]) < 1e-5
