"""Backward passes on pre-activations that left fp16's range: Z is kept in
fp16, so a finite fp32 pre-activation past 65504 comes back as an infinity.
The activations' slopes and values take their limits there (act' 0 and 1,
act(-inf) 0) and only what is infinite itself (act(inf), an infinite up value)
shows as one."""
import numpy as np
import pytest
import torch

import fused_ref as ref
from quantized_linear_layers_token_b200 import synth
from test_gpu_fused import Layer, cuda, host, q, within  # noqa: F401 (q: fixture)

pytestmark = pytest.mark.gpu


def backward(L, act, Z, dY):
    q = L.q  # noqa: F811
    n = (q.qlin_backward_gated_workspace if L.gated else q.qlin_backward_act_workspace)(L.M, L.w)
    dX = torch.full((L.M, L.K), float("nan"), dtype=torch.float16, device="cuda")
    db = torch.full((L.N,), float("nan"), device="cuda")
    (q.qlin_backward_gated if L.gated else q.qlin_backward_act)(L.w, cuda(dY), cuda(Z), L.M, cuda(L.s), dX, db,
                                                                q.empty_workspace(n), n, act=ref.ACTS.index(act))
    q.qlin_poll_device_status()
    return host(dX), host(db)


def inputs(L, share, dy_std):
    """Z with a share of its (gate) entries infinite; what it stands for: the
    slopes are flat long before 65504."""
    rng = np.random.default_rng(L.N)
    Z = rng.standard_normal((L.M, L.N)).astype(np.float16)
    gates = Z[:, 0::2] if L.gated else Z
    minus, plus = rng.random(gates.shape) < share, rng.random(gates.shape) < share
    gates[minus] = -np.inf
    if not L.gated:
        gates[plus] = np.inf
    dY = (rng.standard_normal((L.M, L.Nout)) * dy_std).astype(np.float16)
    return Z, np.clip(Z.astype(np.float64), -65504, 65504), dY


# ring kernels with the mantissas in registers and re-read, the kernel without a ring
@pytest.mark.parametrize("N", [528, 12304, 40000])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ref.ACTS[1:])
def test_limits(q, oracle, act, gated, N):  # noqa: F811
    L = Layer(q, oracle, synth.W8_PERCHANNEL, 21, 128, N, 3, gated=gated)
    Z, z, dY = inputs(L, 0.05, 2.0 ** -7)
    dX, db = backward(L, act, Z, dY)
    dy = dY.astype(np.float64)
    dz, err = ref.dz_gated(dy, z, act) if gated else ref.dz_act(dy, z, act)
    top = (np.abs(dy) * np.maximum(np.abs(z[:, 0::2]), np.abs(z[:, 1::2]))).max(1) if gated else np.abs(dy).max(1)
    want, bound = ref.bias_gradient(dz, err)
    within(db, want, bound + 2.0 ** -120, "dbias")
    want, bound = ref.input_gradient(dz, err, top, L.pk, L.W, L.s)
    within(dX, want, bound, "dX")


@pytest.mark.parametrize("act", ref.ACTS[1:])
def test_small_gradients_keep_their_scale(q, oracle, act):  # noqa: F811
    """An infinite gate does not cost the other channels of its row their
    power of two: with the gradients at 2^-16 and a few channels, dZ in plain
    fp16 would be below its normal range."""
    L = Layer(q, oracle, synth.W8_PERCHANNEL, 9, 128, 64, 0, gated=True)
    Z, z, dY = inputs(L, 0.1, 2.0 ** -16)
    assert np.isinf(Z).any(1).all()
    dX, _ = backward(L, act, Z, dY)
    dy = dY.astype(np.float64)
    dz, err = ref.dz_gated(dy, z, act)
    want, bound = ref.input_gradient(dz, err, (np.abs(dy) * 65504).max(1), L.pk, L.W, L.s)
    within(dX, want, bound, "dX")


@pytest.mark.parametrize("act", ref.ACTS)
def test_overflow_shows(q, oracle, act):  # noqa: F811
    """An infinite activation or up value is an infinity in the gradients of
    its own token and channels, and in no others."""
    L = Layer(q, oracle, synth.W8_PERCHANNEL, 12, 128, 272, 0, gated=True)
    rng = np.random.default_rng(3)
    Z = rng.uniform(0.5, 2, (12, 272)).astype(np.float16)
    dY = np.full((12, 136), 2.0 ** -7, np.float16)
    Z[3, 10] = np.inf   # gate 5: act(inf) reaches up channel 5
    Z[5, 21] = np.inf   # up 10 reaches gate channel 10
    dX, db = backward(L, act, Z, dY)
    bad = ~np.isfinite(dX.astype(np.float32)).all(1)
    assert bad[3] and bad[5] and bad.sum() == 2
    assert np.array_equal(np.flatnonzero(~np.isfinite(db)), [11, 20]) and np.isposinf(db[[11, 20]]).all()


@pytest.mark.parametrize("act", ref.ACTS[1:])
@pytest.mark.parametrize("gated", [False, True])
def test_forward_then_backward(q, oracle, act, gated):  # noqa: F811
    """A training forward whose pre-activations reach -80000: finite outputs,
    and finite gradients from the Z it kept."""
    L = Layer(q, oracle, synth.W8_PERCHANNEL, 20, 128, 64, 0, gated=gated)
    L.bias = np.where(np.arange(64) % 4 == 0, -80000, 0).astype(np.float32)
    L.dXb = cuda(L.bias)
    Z = torch.empty(20, 64, dtype=torch.float16, device="cuda")
    Y, _ = L.forward(act, Z=Z)
    assert torch.isfinite(Y).all() and torch.isneginf(Z[:, 0::4]).all()
    dX, db = backward(L, act, host(Z), np.full((20, L.Nout), 2.0 ** -7, np.float16))
    assert np.isfinite(dX.astype(np.float32)).all() and np.isfinite(db).all() and np.all(db[0::4] == 0)
