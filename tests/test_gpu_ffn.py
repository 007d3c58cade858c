"""The feed-forward block: norm, gated projections, down projection with the
residual, and their backward passes, run together as a model runs them.  Every
stage is held to its 64-bit reference on what the stage before it gave."""
import numpy as np
import pytest
import torch

import fused_ref as ref
from quantized_linear_layers_token_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_linear_layers_token_b200 import qlin
    qlin.lib()
    return qlin


def within(got, want, bound, what):
    got = got.double().cpu().numpy()
    assert np.all(np.isfinite(got)), what
    over = np.abs(got - want) / bound
    assert np.all(over <= 1), (what, float(over.max()))


def h16(t):
    return np.ascontiguousarray(t.cpu().numpy()).view(np.uint16)


class Block:
    def __init__(self, q, oracle, fmt, D, F, nO, kind, bias, seed=0):
        from quantized_linear_layers_token_b200.ffn import GatedFeedForward
        rng = np.random.default_rng([seed, fmt, D, F])
        self.rng, self.oracle, self.fmt = rng, oracle, fmt
        self.Wg = (rng.standard_normal((D, 2 * F)) * 0.03).astype(np.float16)
        self.Wd = (rng.standard_normal((F, D)) * 0.03).astype(np.float16)
        self.Og = np.sort(rng.choice(D, nO, replace=False)).astype(np.int32)
        self.Od = np.sort(rng.choice(F, nO, replace=False)).astype(np.int32)
        c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.c = c
        gated = q.PackedLayer.pack_gated(c(self.Wg[:, 0::2]), c(self.Wg[:, 1::2]), self.Og, fmt)
        down = q.PackedLayer.pack(c(self.Wd), self.Od, fmt)
        self.pg, self.pd = (oracle.pack_layer(w.view(np.uint16), o, fmt) for w, o in ((self.Wg, self.Og), (self.Wd, self.Od)))
        f = lambda n: rng.standard_normal(n).astype(np.float32)  # noqa: E731
        self.gamma, self.beta = 1 + 0.1 * f(D), (0.1 * f(D) if bias else None)
        self.bg, self.bd = (0.2 * f(2 * F), 0.2 * f(D)) if bias else (None, None)
        t = lambda v: None if v is None else c(v)  # noqa: E731
        self.rms = kind == q.QLIN_NORM_RMS
        self.ffn = GatedFeedForward(gated, down, t(self.gamma), t(self.beta), t(self.bg), t(self.bd), kind=kind)

    def x(self, M, D):
        x = self.rng.standard_normal((M, D))
        x[:, self.Og] *= 20
        return x.astype(np.float16)


@pytest.mark.parametrize("fmt", [synth.W4_PERCHANNEL, synth.W4_G128, synth.W8_PERCHANNEL])
@pytest.mark.parametrize("M", [1, 50, 300])
def test_block_forward_and_backward(q, oracle, fmt, M):
    D, F = 512, 640
    kind = q.QLIN_NORM_RMS if M == 50 else q.QLIN_NORM_LAYER
    b = Block(q, oracle, fmt, D, F, 9, kind, bias=M != 50)
    x = b.x(M, D)
    y, saved = b.ffn.forward(b.c(x), training=True)
    dy = (b.rng.standard_normal((M, D)) / 128).astype(np.float16)
    g = b.ffn.backward(saved, b.c(dy))
    q.qlin_poll_device_status()

    # the stages' own results, from the same calls
    n = torch.empty(M, D, dtype=torch.float16, device="cuda")
    q.qlin_norm_forward(b.c(x), M, D, kind, b.ffn.gamma, b.ffn.beta, 1e-5, n)
    want, bound, mu, r, mub, rb = ref.norm_forward(x, b.gamma, b.beta, np.float32(1e-5), b.rms)
    within(n, want, bound, "norm")
    one = np.ones(9, np.float32)
    s = oracle.momentum_update(h16(n), b.Og, b.pg["wmaxO"], 0.9, one)
    assert np.array_equal(saved.s_gated.cpu().numpy(), s)
    z, zerr = ref.preactivation(b.pg, b.Wg, *oracle.quant_act(h16(n), b.Og, s), s, b.bg)
    within(saved.z, z, zerr + ref.H * np.abs(z) + ref.HMIN, "z")
    h = torch.empty(M, F, dtype=torch.float16, device="cuda")
    ws = q.qlin_forward_gated_workspace(M, b.ffn.gated.w)
    q.qlin_forward_gated(n, M, b.ffn.gated.w, b.c(s), 0.9, False, h, q.empty_workspace(ws), ws, bias=b.ffn.bias_gated)
    within(h, *ref.forward_gated(z, zerr, "silu"), "h")
    sd = oracle.momentum_update(h16(h), b.Od, b.pd["wmaxO"], 0.9, one)
    assert np.array_equal(saved.s_down.cpu().numpy(), sd)
    zd, zderr = ref.preactivation(b.pd, b.Wd, *oracle.quant_act(h16(h), b.Od, sd), sd, b.bd)
    within(y, *ref.forward_act(zd, zderr, "none", x), "y")

    # backward, stage by stage
    d64 = dy.astype(np.float64)
    dh = torch.empty(M, F, dtype=torch.float16, device="cuda")
    dn = torch.empty(M, D, dtype=torch.float16, device="cuda")
    ws = max(q.qlin_backward_act_workspace(M, b.ffn.down.w), q.qlin_backward_gated_workspace(M, b.ffn.gated.w))
    buf = q.empty_workspace(ws)
    q.qlin_backward_act(b.ffn.down.w, b.c(dy), None, M, saved.s_down, dh, None, buf, ws)
    within(dh, *ref.input_gradient(d64, 0 * d64, np.abs(d64).max(1), b.pd, b.Wd, sd), "dh")
    q.qlin_backward_gated(b.ffn.gated.w, dh, saved.z, M, saved.s_gated, dn, None, buf, ws)
    zz, hh = saved.z.double().cpu().numpy(), dh.double().cpu().numpy()
    dz, err = ref.dz_gated(hh, zz, "silu")
    top = (np.abs(hh) * np.maximum(np.abs(zz[:, 0::2]), np.abs(zz[:, 1::2]))).max(1)
    within(dn, *ref.input_gradient(dz, err, top, b.pg, b.Wg, s), "dn")
    out = ref.norm_backward(dn.cpu().numpy(), x, b.gamma, None if b.rms else saved.mean.cpu().numpy(),
                            saved.rstd.cpu().numpy(), dy, b.rms)
    within(g["dx"], out[0], out[1], "dx")
    within(g["dgamma"], out[2], out[3] + 1e-30, "dgamma")
    if b.beta is None:
        assert g["dbeta"] is None and g["dbias_gated"] is None and g["dbias_down"] is None
    else:
        within(g["dbeta"], out[4], out[5] + 1e-30, "dbeta")
        want, bound = ref.bias_gradient(dz, err)
        within(g["dbias_gated"], want, bound + 1e-30, "dbias_gated")
        want, bound = ref.bias_gradient(d64, 0 * d64)
        within(g["dbias_down"], want, bound + 1e-30, "dbias_down")


def test_block_token_counts_in_turn(q, oracle):
    """One object over changing token counts, with a backward pass between:
    each result is that of a fresh object."""
    b = Block(q, oracle, synth.W4_G128, 256, 384, 5, q.QLIN_NORM_RMS, bias=False)
    xs = {M: b.c(b.x(M, 256)) for M in (1, 40, 3, 600, 40)}
    fresh = {}
    for M, x in xs.items():
        f = Block(q, oracle, synth.W4_G128, 256, 384, 5, q.QLIN_NORM_RMS, bias=False)
        fresh[M] = f.ffn.forward(x)
    for M in (1, 40, 3, 600, 40, 1, 600, 600):
        assert torch.equal(b.ffn.forward(xs[M]), fresh[M]), M
        if M > 1:
            # a training step on the side, its momentum taken back
            keep = b.ffn.s_gated.clone(), b.ffn.s_down.clone()
            y, saved = b.ffn.forward(xs[M], training=True)
            b.ffn.backward(saved, y)
            b.ffn.s_gated.copy_(keep[0])
            b.ffn.s_down.copy_(keep[1])
    q.qlin_poll_device_status()


def test_block_training_step_in_a_graph(q, oracle):
    """Forward and backward captured once, replayed on new inputs: the eager
    results, bit for bit."""
    b = Block(q, oracle, synth.W8_PERCHANNEL, 256, 384, 5, q.QLIN_NORM_LAYER, bias=True)
    x, dy = b.c(b.x(64, 256)), b.c((b.rng.standard_normal((64, 256)) / 64).astype(np.float16))
    s0 = b.ffn.s_gated.clone(), b.ffn.s_down.clone()

    def step():
        y, saved = b.ffn.forward(x, training=True)
        g = b.ffn.backward(saved, dy)
        return [y, saved.s_gated, saved.s_down, *(g[k] for k in sorted(g))]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        x.copy_(torch.randn(64, 256, device="cuda"))
        if k:  # other token counts in between, and memory that is reused
            for M in (3, 200):
                y, saved = b.ffn.forward(b.c(b.x(M, 256)), training=True)
                b.ffn.backward(saved, y)
            torch.empty(1 << 26, dtype=torch.uint8, device="cuda").fill_(255)
        b.ffn.s_gated.copy_(s0[0])
        b.ffn.s_down.copy_(s0[1])
        graph.replay()
        got = [t.clone() for t in out]
        b.ffn.s_gated.copy_(s0[0])
        b.ffn.s_down.copy_(s0[1])
        for a, c in zip(got, step()):
            assert torch.equal(a, c)


def test_block_refuses_layers_that_do_not_fit(q):
    from quantized_linear_layers_token_b200.ffn import GatedFeedForward
    gated = q.PackedLayer(256, 512, synth.W8_PERCHANNEL, 0)
    with pytest.raises(ValueError):
        GatedFeedForward(gated, q.PackedLayer(512, 256, synth.W8_PERCHANNEL, 0), torch.ones(256, device="cuda"))


def test_block_captured_at_a_new_token_count(q, oracle):
    """Captured without an eager call of that token count before, then called
    eagerly and replayed, in either order, and captured twice: one result."""
    make = lambda: Block(q, oracle, synth.W4_G128, 256, 384, 5, q.QLIN_NORM_RMS, bias=False)  # noqa: E731
    x = make().c(make().x(300, 256))
    want = make().ffn.forward(x)
    for eager_first in (True, False):
        b = make()
        b.ffn.forward(x[:7])
        graphs, outs = [], []
        junk = torch.empty(1 << 26, dtype=torch.uint8, device="cuda").fill_(255)
        del junk
        for _ in range(2):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                outs.append(b.ffn.forward(x))
        if eager_first:
            assert torch.equal(b.ffn.forward(x), want)
        for k in (1, 0, 1):
            outs[k].zero_()
            graphs[k].replay()
            assert torch.equal(outs[k], want), k
        assert torch.equal(b.ffn.forward(x), want)
    q.qlin_poll_device_status()


def test_block_refuses_other_shapes(q, oracle):
    """A padded batch, another width, or gradients of another token count."""
    b = Block(q, oracle, synth.W8_PERCHANNEL, 256, 384, 0, q.QLIN_NORM_RMS, bias=False)
    x = b.c(b.x(6, 256))
    for bad in (x.view(2, 3, 256), x.view(3, 512), x.view(12, 128), x.t(), x.float(), x.cpu()):
        with pytest.raises(ValueError):
            b.ffn.forward(bad)
    y, saved = b.ffn.forward(x, training=True)
    for bad in (y[:5], y.view(2, 3, 256), y.float()):
        with pytest.raises(ValueError):
            b.ffn.backward(saved, bad)
    assert b.ffn.forward(x[:0]).shape == (0, 256)
