"""64-bit references of the fused layers and norms, and the bounds their
kernels are held to.  Plain numpy; codes and packed weights come from the
oracle.

Roundings counted in the bounds (halves of a step, relative): fp16 2^-11 (and
2^-25 absolute below its normal range), fp32 2^-24."""
import math

import numpy as np
import torch

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")  # codes 0 .. 4
H = 2.0 ** -11       # one rounding to fp16
HMIN = 2.0 ** -25    # ... below its normal range
# the fp32 exponential is documented to 2 + |1.173 x| units of 2^-23 at most:
# 2^-17 covers |x| <= 50, past which exp(-x) is below 2^-72; quotients,
# products and the normal distribution's few units are far below that
APPROX = 2.0 ** -17


def phi(z):
    t = torch.from_numpy(np.ascontiguousarray(z))
    return (0.5 * torch.special.erfc(-t / math.sqrt(2.0))).numpy()


def act(name, z):
    """(act(z), act'(z)) in fp64."""
    if name == "none":
        return z.copy(), np.ones_like(z)
    if name == "relu":
        return np.maximum(z, 0.0), (z > 0).astype(np.float64)
    if name == "gelu":
        p = phi(z)
        return z * p, p + z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        t = np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 0.134145 * z * z)
    with np.errstate(over="ignore"):
        p = 1 / (1 + np.exp(-z))
    return z * p, p + z * p * (1 - p)


def preactivation(pk, W, Xq, a, XqO, s, bias):
    """Z in fp64 and the bound of its fp32 evaluation: the sum of the integer
    product is exact, the compensation's products carry 2^-21 each (two fp16
    terms) and are added in fp32, three more fp32 operations follow."""
    q = Xq.astype(np.float64)
    cs = pk["cscale"].astype(np.float64)
    main = (q @ pk["B"].astype(np.float64)) * cs
    ad = a.astype(np.float64)[:, None]
    O = pk["O"]
    u = XqO.astype(np.float64) * (s.astype(np.float64) - 1.0)
    WO = W[O].astype(np.float64)
    comp, mag = u @ WO, np.abs(u) @ np.abs(WO)
    b = np.zeros(W.shape[1]) if bias is None else bias.astype(np.float64)
    z = ad * (main + comp) + b
    err = ad * (np.abs(main) * 2.0 ** -22 + mag * (2.0 ** -20 + len(O) * 2.0 ** -22)) + (np.abs(z) + np.abs(b)) * 2.0 ** -23
    return z, err


def forward_act(z, zerr, name, residual):
    """Y of the layer with an epilogue and its bound (|act'| <= 1.13)."""
    v, _ = act(name, z)
    r = 0.0 if residual is None else residual.astype(np.float64)
    y = v + r
    return y, 1.13 * zerr + APPROX * np.abs(v) + 2.0 ** -24 * np.abs(y) + H * np.abs(y) + HMIN


def forward_gated(z, zerr, name):
    g, u = z[:, 0::2], z[:, 1::2]
    v, _ = act(name, g)
    y = v * u
    bound = np.abs(u) * (1.13 * zerr[:, 0::2] + APPROX * np.abs(v)) + 1.01 * np.abs(v) * zerr[:, 1::2]
    return y, bound + 2.0 ** -23 * np.abs(y) + H * np.abs(y) + HMIN


def dz_act(dy, z, name):
    """dZ and the bound of its fp32 evaluation (the slope's terms may cancel)."""
    _, d = act(name, z)
    return dy * d, np.abs(dy) * APPROX * (1 + np.abs(z) * (z > -30) * (z < 30))


def dz_gated(dh, z, name):
    g, u = z[:, 0::2], z[:, 1::2]
    v, d = act(name, g)
    dz, err = np.empty_like(z), np.empty_like(z)
    dz[:, 0::2], dz[:, 1::2] = dh * u * d, dh * v
    err[:, 0::2] = np.abs(dh * u) * APPROX * (1 + np.abs(g) * (np.abs(g) < 30))
    err[:, 1::2] = np.abs(dh * v) * APPROX
    return dz, err


def input_gradient(dz, err, top, pk, W, s):
    """dX and its bound.  dZ is rounded to fp16 once, in a row scaled so that
    `top` (the row's largest possible |dZ|) lies in [2^13, 2^14): 2^-11 of
    the value, or 2^-25 2^-13 of 2 top below the normal range; the outlier
    rows of Weff are rounded to fp16; N fp32 additions; one rounding."""
    Wd = pk["B"].astype(np.float64) * pk["cscale"].astype(np.float64)[None, :]
    We, mag = Wd.copy(), np.abs(Wd)
    rnd = np.zeros_like(Wd)
    O = pk["O"]
    if len(O):
        sd = s.astype(np.float64)[:, None]
        WO = W[O].astype(np.float64)
        We[O] = (Wd[O] + (sd - 1.0) * WO) / sd
        mag[O] = (np.abs(Wd[O]) + np.abs(sd - 1.0) * np.abs(WO)) / sd
        rnd[O] = np.abs(We[O]) * H + mag[O] * 2.0 ** -22
    N = dz.shape[1]
    dx = dz @ We.T
    adz = np.abs(dz)
    each = adz * (H + 2.0 ** -22) + err + top[:, None] * 2.0 ** -37
    bound = each @ mag.T + adz @ rnd.T + (adz @ mag.T) * N * 2.0 ** -22 + np.abs(dx) * H + HMIN
    return dx, bound


def bias_gradient(dz, err):
    """dbias and its bound: M fp32 additions."""
    return dz.sum(0), np.abs(dz).sum(0) * (dz.shape[0] + 1) * 2.0 ** -24 + err.sum(0)


# A row's fp32 sums: at most 64 values a thread, then a tree over at most
# 1024 threads in 15 steps: 79 additions in a chain, below 2^-17 of the sum
# of magnitudes.
ROW = 2.0 ** -17


def norm_forward(x, gamma, beta, eps, rms):
    x, g = x.astype(np.float64), gamma.astype(np.float64)
    b = np.zeros_like(g) if beta is None else beta.astype(np.float64)
    mu = np.zeros((x.shape[0], 1)) if rms else x.mean(1, keepdims=True)
    r = 1 / np.sqrt(((x - mu) ** 2).mean(1, keepdims=True) + eps)
    y = (x - mu) * r * g + b
    mu_err = 0.0 if rms else ROW * np.abs(x).mean(1, keepdims=True)
    # r: half the relative error of the mean square, which an error of mu
    # enters squared only, and a few fp32 operations
    r_rel = ROW + (mu_err * r) ** 2
    bound = np.abs(g) * r * mu_err + np.abs((x - mu) * r * g) * (r_rel + 2.0 ** -21) + 2.0 ** -23 * np.abs(y)
    return y, bound + H * np.abs(y) + HMIN, mu[:, 0], r[:, 0], (mu_err + 0 * r)[:, 0], (r * r_rel)[:, 0]


def norm_backward(dy, x, gamma, mean, rstd, dres, rms):
    x, dy, g = x.astype(np.float64), dy.astype(np.float64), gamma.astype(np.float64)
    mu = np.zeros((x.shape[0], 1)) if rms else mean.astype(np.float64)[:, None]
    r = rstd.astype(np.float64)[:, None]
    xh = (x - mu) * r
    w = dy * g
    m1 = 0.0 if rms else w.mean(1, keepdims=True)
    m2 = (w * xh).mean(1, keepdims=True)
    core = w - m1 - xh * m2
    dx = r * core + (0.0 if dres is None else dres.astype(np.float64))
    aw = np.abs(w)
    err = r * (ROW * (aw.mean(1, keepdims=True) * (not rms) + np.abs(xh) * (aw * np.abs(xh)).mean(1, keepdims=True))
               + 2.0 ** -21 * (aw + np.abs(xh * m2) + np.abs(m1)))
    bound = err + 2.0 ** -23 * np.abs(dx) + H * np.abs(dx) + HMIN
    t = dy * xh
    M = x.shape[0]
    # M additions and three products or sums in each term
    dg, dg_b = t.sum(0), np.abs(t).sum(0) * (M + 4) * 2.0 ** -24
    db, db_b = dy.sum(0), np.abs(dy).sum(0) * (M + 1) * 2.0 ** -24
    return dx, bound, dg, dg_b, db, db_b
