"""Gradients that are zero but in a few channels, for sharp checks of the input
gradient of wide layers: a sum over all channels has a worst-case rounding bound
that grows with their number and hides a lost step, a sum of a few terms does
not (adding zeros is exact)."""
import numpy as np

import fused_ref as ref


def channels(N, rng):
    """The first vector of 8, the last vector, the first vector of the last
    64-channel step, and eight more anywhere."""
    last = (N - 1) // 64 * 64
    fixed = [np.arange(8), np.arange(N - 8, N), np.arange(last, last + 8)]
    return np.unique(np.concatenate([*fixed, rng.choice(N, 8, replace=False)]))


def gradient(M, N, gated, rng, std=2.0 ** -7):
    """(dY, the channels of Z that it reaches)."""
    cols = channels(N, rng)
    if gated:
        cols = np.unique(cols // 2)
        dY = np.zeros((M, N // 2), np.float16)
        dY[:, cols] = (rng.standard_normal((M, len(cols))) * std).astype(np.float16)
        return dY, np.stack([2 * cols, 2 * cols + 1], 1).reshape(-1)
    dY = np.zeros((M, N), np.float16)
    dY[:, cols] = (rng.standard_normal((M, len(cols))) * std).astype(np.float16)
    return dY, cols


def reference(act, gated, dY, Z, at, pk, W, s):
    """(dZ of the channels `at`, dX and its bound): the layer of these channels alone."""
    z = Z[:, at].astype(np.float64)
    if gated:
        dy = dY[:, at[0::2] // 2].astype(np.float64)
        dz, err = ref.dz_gated(dy, z, act)
        top = (np.abs(dy) * np.maximum(np.abs(z[:, 0::2]), np.abs(z[:, 1::2]))).max(1)
    else:
        dy = dY[:, at].astype(np.float64)
        dz, err = ref.dz_act(dy, z, act)
        top = np.abs(dy).max(1)
    part = {"B": pk["B"][:, at], "cscale": pk["cscale"][at], "O": pk["O"]}
    return dz, *ref.input_gradient(dz, err, top, part, W[:, at], s)
