"""One workspace, zero-filled once, under every call that takes one: layers,
token counts and entry points in any order give the bits that each gives on a
fresh zero-filled workspace."""
import random

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


class Layer:
    def __init__(self, q, fmt, K, N, nO, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
        O = np.sort(np.random.default_rng(seed).choice(K, nO, replace=False)).astype(np.int32)
        self.layer = q.PackedLayer.pack((self.n(K, N) * 0.02).half(), O, fmt)
        self.w, self.K, self.N, self.s = self.layer.w, K, N, 1 + 3 * torch.rand(nO, generator=gen, device="cuda")


def half(*shape):
    return torch.full(shape, float("nan"), dtype=torch.float16, device="cuda")


def forward(q, L, M, update):
    X = L.n(M, L.K).half()

    def call(ws):
        Y, s = half(M, L.N), L.s.clone()
        q.qlin_forward(X, M, L.w, s, 0.9, update, Y, ws, ws.numel())
        return [Y, s]
    return q.qlin_forward_workspace(M, L.w), call


def forward_fused(q, L, M, gated, update):
    X, R = L.n(M, L.K).half(), L.n(M, L.N).half()

    def call(ws):
        Y, s = half(M, L.N // 2 if gated else L.N), L.s.clone()
        if gated:
            q.qlin_forward_gated(X, M, L.w, s, 0.9, update, Y, ws, ws.numel())
        else:
            q.qlin_forward_act(X, M, L.w, s, 0.9, update, Y, ws, ws.numel(), act=4, residual=R)
        return [Y, s]
    size = q.qlin_forward_gated_workspace if gated else q.qlin_forward_act_workspace
    return size(M, L.w), call


def quant_and_gemm(q, L, M):
    X = L.n(M, L.K).half()

    def call(ws):
        s, a = L.s.clone(), torch.empty(M, device="cuda")
        Xq = torch.empty(M, L.K, dtype=torch.int8, device="cuda")
        XqO = torch.empty(M, max(len(L.s), 1), dtype=torch.int8, device="cuda")
        Y = half(M, L.N)
        q.qlin_quant_act(X, M, L.w, s, 0.9, True, Xq, a, XqO, ws, ws.numel())
        q.qlin_gemm(L.w, Xq, a, XqO, s, M, Y, None, ws, ws.numel())
        return [Y, s, Xq]
    return max(q.qlin_quant_act_workspace(M, L.w), q.qlin_gemm_workspace(M, L.w)), call


def grouped(q, Ls, M):
    Xs = [L.n(M, L.K).half() for L in Ls]

    def call(ws):
        Ys, ss = [half(M, L.N) for L in Ls], [L.s.clone() for L in Ls]
        q.qlin_forward_grouped([L.w for L in Ls], Xs, ss, Ys, M, 0.9, True, ws, ws.numel())
        return Ys + ss
    return q.qlin_forward_grouped_workspace([L.w for L in Ls], M), call


def backward_dx(q, L, M):
    dY = (L.n(M, L.N) / 128).half()

    def call(ws):
        dX = half(M, L.K)
        q.qlin_backward_dx(L.w, dY, M, L.s, dX, ws, ws.numel())
        return [dX]
    return q.qlin_backward_dx_workspace(M, L.w), call


def backward_fused(q, L, M, gated):
    dY, Z = (L.n(M, L.N // 2 if gated else L.N) / 128).half(), L.n(M, L.N).half()

    def call(ws):
        dX, db = half(M, L.K), torch.empty(L.N, device="cuda")
        (q.qlin_backward_gated if gated else q.qlin_backward_act)(L.w, dY, Z, M, L.s, dX, db, ws, ws.numel(), act=4)
        return [dX, db]
    size = q.qlin_backward_gated_workspace if gated else q.qlin_backward_act_workspace
    return size(M, L.w), call


def norm_backward(q, M, K):
    gen = torch.Generator(device="cuda").manual_seed(K)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    X, dY, gamma, mean, rstd = n(M, K).half(), (n(M, K) / 128).half(), n(K), 0.1 * n(M), 1 + 0.1 * n(M)

    def call(ws):
        dX, dg, db = half(M, K), torch.empty(K, device="cuda"), torch.empty(K, device="cuda")
        q.qlin_norm_backward(dY, X, M, K, q.QLIN_NORM_LAYER, gamma, mean, rstd, None, dX, dg, db, ws, ws.numel())
        return [dX, dg, db]
    return q.qlin_norm_backward_workspace(M, K), call


def calls(q, kinds):
    pc, g128, w8 = synth.W4_PERCHANNEL, synth.W4_G128, synth.W8_PERCHANNEL
    Ls = [Layer(q, pc, 2048, 528, 40, 1), Layer(q, g128, 1024, 2064, 7, 2), Layer(q, w8, 4096, 272, 90, 3),
          Layer(q, w8, 512, 656, 0, 4)]
    out = []
    for i, L in enumerate(Ls):
        for M in (1, 16, 40, 70, 130, 300, 700):
            if "fused" in kinds:
                out += [forward_fused(q, L, M, False, i % 2 == 0), forward_fused(q, L, M, True, i % 2 == 1)]
            if "layer" in kinds:
                out += [forward(q, L, M, True), quant_and_gemm(q, L, M)]
            if "backward" in kinds and M in (16, 300, 700):
                out += [backward_dx(q, L, M), backward_fused(q, L, M, False), backward_fused(q, L, M, True)]
    if "layer" in kinds:
        four = [Layer(q, pc, K, N, nO, K + N) for K, N, nO in ((1024, 272, 9), (512, 1040, 0), (2048, 400, 33))]
        out += [grouped(q, four, M) for M in (1, 16, 48)]
    if "backward" in kinds:
        out += [norm_backward(q, M, K) for M, K in ((5, 512), (700, 4096), (300, 20000))]
    return out


@pytest.mark.parametrize("knobs", [{}, {"fused_momentum_max_m": 0}, {"pair_split": 1}, {"cluster": 0}], ids=str)
@pytest.mark.parametrize("kinds", [("fused",), ("fused", "layer"), ("fused", "layer", "backward")], ids="+".join)
def test_shared_workspace(q, kinds, knobs):
    with q.knobs(**knobs):
        todo = calls(q, kinds)
        want = [call(q.empty_workspace(n)) for n, call in todo]
        ws = q.empty_workspace(max(n for n, _ in todo))
        order = random.Random(7)
        for _ in range(3):
            for k in order.sample(range(len(todo)), len(todo)):
                for a, b in zip(todo[k][1](ws), want[k]):
                    assert torch.equal(a, b), (k, todo[k][0])
    q.qlin_poll_device_status()
