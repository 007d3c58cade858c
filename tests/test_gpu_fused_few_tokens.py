"""Input gradients of up to 128 tokens: dZ goes into the product as two fp16
terms, so what is left beside the last rounding of dX is far below it.  (With
few tokens the gradient has few numbers, and the rounding of each shows.)"""
import numpy as np
import pytest
import torch

import fused_ref as ref
import sparse_gradient as sparse
from quantized_linear_layers_token_b200 import synth
from test_gpu_fused import FMTS, Layer, cuda, host, q, within  # noqa: F401 (q: fixture)

pytestmark = pytest.mark.gpu


def backward(L, act, Z, dY, dbias=False):
    q = L.q  # noqa: F811
    dX = torch.full((L.M + 2, L.K), float("nan"), dtype=torch.float16, device="cuda")
    db = torch.empty(L.N, device="cuda") if dbias else None
    n = (q.qlin_backward_gated_workspace if L.gated else q.qlin_backward_act_workspace)(L.M, L.w)
    ws = q.empty_workspace(n)
    ws[q.QLIN_WORKSPACE_HEAD:].fill_(255)
    call = q.qlin_backward_gated if L.gated else q.qlin_backward_act
    got = []
    for _ in range(2):
        call(L.w, cuda(dY), cuda(Z), L.M, cuda(L.s), dX, db, ws, n, act=ref.ACTS.index(act))
        got.append(dX.clone())
    q.qlin_poll_device_status()
    assert torch.equal(got[0][:L.M].view(torch.int16), got[1][:L.M].view(torch.int16)) and torch.isnan(dX[L.M:]).all()
    assert (ws[:q.QLIN_WORKSPACE_HEAD] == 0).all()
    return host(dX[:L.M])


def two_term_bound(dz, err, top, B, cscale, O, W, s, dx):
    """Roundings: dZ in two fp16 terms and two fp32 products (2^-21, or 2^-37 of
    the row's bound below fp16's normal range), outlier rows 2^-11, one fp32
    addition a term and term of dZ, one rounding of dX."""
    Wd = B.astype(np.float64) * cscale.astype(np.float64)[None, :]
    mag, rnd = np.abs(Wd), np.zeros_like(Wd)
    if len(O):
        sd, WO = s.astype(np.float64)[:, None], W[O].astype(np.float64)
        mag[O] = (np.abs(Wd[O]) + np.abs(sd - 1) * np.abs(WO)) / sd
        rnd[O] = np.abs((Wd[O] + (sd - 1) * WO) / sd) * ref.H + mag[O] * 2.0 ** -22
    adz = np.abs(dz)
    each = adz * 2.0 ** -21 + err + top[:, None] * 2.0 ** -37
    return each @ mag.T + adz @ rnd.T + (adz @ mag.T) * dz.shape[1] * 2.0 ** -22 + np.abs(dx) * ref.H + ref.HMIN


# one and several ranges of the reduction, ragged channels, both kernels of the activation
@pytest.mark.parametrize("N", [272, 4112, 40000])
@pytest.mark.parametrize("M", [1, 2, 31, 127, 128])
@pytest.mark.parametrize("gated", [False, True])
def test_each_element(q, oracle, gated, M, N):  # noqa: F811
    fmt = FMTS[(M + N) % 3]
    L = Layer(q, oracle, fmt, M, 384, N, 5, gated=gated)
    rng = np.random.default_rng([M, N])
    Z = (rng.standard_normal((M, N)) * 1.5).astype(np.float16)
    dY, at = sparse.gradient(M, N, gated, rng)
    act = "relu" if gated else "none"
    dz, want, _ = sparse.reference(act, gated, dY, Z, at, L.pk, L.W, L.s)
    z, dy = Z[:, at].astype(np.float64), np.abs(dY.astype(np.float64))
    top = (dy[:, at[0::2] // 2] * np.maximum(np.abs(z[:, 0::2]), np.abs(z[:, 1::2]))).max(1) if gated else dy.max(1)
    bound = two_term_bound(dz, 0 * dz, top, L.pk["B"][:, at], L.pk["cscale"][at], L.pk["O"], L.W[:, at], L.s, want)
    within(backward(L, act, Z, dY, dbias=M % 2 == 0), want, bound, "dX")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [3, 40, 128])
def test_error_is_the_last_rounding(q, oracle, fmt, M):  # noqa: F811
    """In the 2-norm: dense gradients, every activation's slope; beside one
    rounding to fp16 the rest (2^-21 a term, the slopes' 2^-17) is below a tenth."""
    L = Layer(q, oracle, fmt, M, 640, 2064, 0, gated=True)
    rng = np.random.default_rng(M)
    Z = rng.standard_normal((M, 2064)).astype(np.float16)
    dY = (rng.standard_normal((M, 1032)) / 128).astype(np.float16)
    for act in ref.ACTS:
        got = backward(L, act, Z, dY).astype(np.float64)
        dz, _ = ref.dz_gated(dY.astype(np.float64), Z.astype(np.float64), act)
        want = dz @ (L.pk["B"].astype(np.float64) * L.pk["cscale"].astype(np.float64)[None, :]).T
        once = np.linalg.norm(want.astype(np.float16).astype(np.float64) - want)
        assert np.linalg.norm(got - want) <= 1.1 * once, act


@pytest.mark.parametrize("M", [1, 128])
def test_infinite_gradient_shows(q, oracle, M):  # noqa: F811
    L = Layer(q, oracle, synth.W8_PERCHANNEL, M, 128, 256, 0)
    dY = np.full((M, 256), 2.0 ** -7, np.float16)
    dY[M // 2, 100] = np.inf
    bad = ~np.isfinite(backward(L, "none", np.zeros((M, 256), np.float16), dY).astype(np.float32)).all(1)
    assert bad[M // 2] and bad.sum() == 1


@pytest.mark.parametrize("dy_std", [3e-7, 2.0 ** -7, 3000.0])
def test_gradient_scales(q, oracle, dy_std):  # noqa: F811
    L = Layer(q, oracle, synth.W8_PERCHANNEL, 33, 256, 512, 0, gated=True)
    rng = np.random.default_rng(5)
    Z = rng.standard_normal((33, 512)).astype(np.float16)
    dY = (rng.standard_normal((33, 256)) * dy_std).astype(np.float16)
    got = backward(L, "relu", Z, dY).astype(np.float64)
    dz, _ = ref.dz_gated(dY.astype(np.float64), Z.astype(np.float64), "relu")
    want = dz @ (L.pk["B"].astype(np.float64) * L.pk["cscale"].astype(np.float64)[None, :]).T
    once = want.astype(np.float16).astype(np.float64)
    fit = np.isfinite(once)
    assert np.array_equal(np.isfinite(got), fit)
    assert np.linalg.norm((got - want)[fit]) <= 1.1 * np.linalg.norm((once - want)[fit])
