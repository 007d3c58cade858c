"""GPU parity of the layers with a fused epilogue (bias, activation, residual),
of the gated block, and of their backward passes, against 64-bit references
(fused_ref.py) on the oracle's codes."""
import numpy as np
import pytest
import torch

import fused_ref as ref
from quantized_linear_layers_token_b200 import synth

pytestmark = pytest.mark.gpu
FMTS = [synth.W4_PERCHANNEL, synth.W4_G128, synth.W8_PERCHANNEL]
GAMMA = 0.9


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_linear_layers_token_b200 import qlin
    qlin.lib()
    return qlin


def cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.cpu().numpy()


def ws_for(q, n):
    return q.empty_workspace(n), n


class Layer:
    """One layer (gated: W's even channels are the gate) with its inputs."""

    def __init__(self, q, oracle, fmt, M, K, N, nO, gated=False, bias=True, residual=True, seed=0):
        rng = np.random.default_rng([seed, fmt, M, K, N, nO])
        self.q, self.M, self.K, self.N, self.gated = q, M, K, N, gated
        self.O = np.sort(rng.choice(K, nO, replace=False)).astype(np.int32)
        self.W = (rng.standard_normal((K, N)) * 0.02).astype(np.float16)
        x = rng.standard_normal((M, K))
        x[:, self.O] *= rng.uniform(20, 60, nO)
        self.X = x.astype(np.float16)
        self.s = rng.uniform(1, 8, nO).astype(np.float32)
        self.bias = (0.3 * rng.standard_normal(N)).astype(np.float32) if bias else None
        self.res = rng.standard_normal((M, N)).astype(np.float16) if residual and not gated else None
        self.pk = oracle.pack_layer(self.W.view(np.uint16), self.O, fmt)
        self.oracle = oracle
        if gated:
            self.layer = q.PackedLayer.pack_gated(cuda(self.W[:, 0::2]), cuda(self.W[:, 1::2]), self.O, fmt)
        else:
            self.layer = q.PackedLayer.pack(cuda(self.W), self.O, fmt)
        self.w = self.layer.w
        self.Nout = N // 2 if gated else N
        self.dX, self.dXb = cuda(self.X), cuda(self.bias)
        size = q.qlin_forward_gated_workspace if gated else q.qlin_forward_act_workspace
        self.ws, self.nws = ws_for(q, size(M, self.w))

    def forward(self, act, update=False, Z=None, s=None, Y=None, res="own", stream=None):
        q = self.q
        Y = torch.full((self.M, self.Nout), float("nan"), dtype=torch.float16, device="cuda") if Y is None else Y
        s = cuda(self.s) if s is None else s
        kw = dict(act=ref.ACTS.index(act), bias=self.dXb, Z=Z, stream=stream)
        if self.gated:
            q.qlin_forward_gated(self.dX, self.M, self.w, s, GAMMA, update, Y, self.ws, self.nws, **kw)
        else:
            kw["residual"] = cuda(self.res) if isinstance(res, str) else res
            q.qlin_forward_act(self.dX, self.M, self.w, s, GAMMA, update, Y, self.ws, self.nws, **kw)
        return Y, s

    def reference(self, act, s):
        Xq, a, XqO = self.oracle.quant_act(self.X.view(np.uint16), self.O, s)
        z, zerr = ref.preactivation(self.pk, self.W, Xq, a, XqO, s, self.bias)
        y, bound = ref.forward_gated(z, zerr, act) if self.gated else ref.forward_act(z, zerr, act, self.res)
        return z, zerr, y, bound


def within(got, want, bound, what):
    """Within the bound; a value that rounds past fp16's largest finite one
    (|want| >= 65520, half a step above 65504, give or take the bound) may be,
    and beyond the bound has to be, the infinity of its sign."""
    got = got.astype(np.float64)
    past = (np.abs(want) + bound >= 65520) & (got == np.copysign(np.inf, want))
    assert np.all(np.isfinite(got) | past), what
    over = np.where(past, 0, np.abs(got - want)) / bound
    assert np.all(over <= 1), (what, float(over.max()), np.unravel_index(over.argmax(), over.shape))


def check_forward(L, act, update=False, keep_z=False):
    Z = torch.full((L.M, L.N), float("nan"), dtype=torch.float16, device="cuda") if keep_z else None
    Y, s = L.forward(act, update, Z)
    L.q.qlin_poll_device_status()
    s1 = L.s
    if update and len(L.O):
        s1 = L.oracle.momentum_update(L.X.view(np.uint16), L.O, L.pk["wmaxO"], GAMMA, L.s)
        assert np.array_equal(host(s).view(np.uint32), s1.view(np.uint32))
    z, zerr, y, bound = L.reference(act, s1)
    within(host(Y), y, bound, "Y")
    if keep_z:
        within(host(Z), z, zerr + ref.H * np.abs(z) + ref.HMIN, "Z")
    return Y


# one token (cluster split-K), every token tile, ragged tokens and channels,
# inputs short of a block, CTA pairs, INT4 widened once per call
SHAPES = [(1, 512, 256, 10), (16, 1152, 2064, 23), (31, 128, 16, 0), (64, 384, 144, 5), (67, 1152, 1040, 21),
          (130, 512, 400, 70), (300, 1024, 272, 16), (513, 256, 528, 5), (700, 2176, 656, 40)]


@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)))
@pytest.mark.parametrize("fmt", FMTS)
def test_forward_act(q, oracle, fmt, i, shape):
    L = Layer(q, oracle, fmt, *shape, bias=i % 3 != 2, residual=i % 2 == 0)
    check_forward(L, ref.ACTS[(i + fmt) % 5], update=i % 2 == 1, keep_z=i % 3 != 1)
    check_forward(L, "none")  # the workspace is left ready


@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)))
@pytest.mark.parametrize("fmt", FMTS)
def test_forward_gated(q, oracle, fmt, i, shape):
    L = Layer(q, oracle, fmt, *shape, gated=True, bias=i % 2 == 0)
    check_forward(L, ref.ACTS[1 + (i + fmt) % 4], update=i % 2 == 0, keep_z=i % 3 != 0)
    check_forward(L, "silu", keep_z=True)


@pytest.mark.parametrize("K", [32, 96, 1056])
def test_forward_short_inputs(q, oracle, K):
    """K that is not a multiple of the 128-wide block (INT8 and per-channel INT4)."""
    for fmt in (synth.W4_PERCHANNEL, synth.W8_PERCHANNEL):
        for M in (5, 300):
            check_forward(Layer(q, oracle, fmt, M, K, 176, 3), "gelu", keep_z=True)
            check_forward(Layer(q, oracle, fmt, M, K, 176, 3, gated=True), "gelu_tanh", keep_z=True)


@pytest.mark.parametrize("fmt", FMTS)
def test_long_inputs(q, oracle, fmt):
    """Few tiles of many inputs: every token tile cut into ranges."""
    for M in (1, 20, 60, 100, 200):
        for gated in (False, True):
            check_forward(Layer(q, oracle, fmt, M, 8192, 272, 40, gated=gated), "silu", keep_z=True)


@pytest.mark.parametrize("act", ref.ACTS)
def test_every_activation(q, oracle, act):
    """Each activation in each of the four epilogues: cluster split-K,
    stream-K, whole tiles and CTA pairs."""
    for M, knobs in [(4, {}), (40, {"cluster": 0}), (20, {"max_ctas": 1}), (300, {})]:
        with q.knobs(**knobs):
            for gated in (False, True):
                check_forward(Layer(q, oracle, synth.W8_PERCHANNEL, M, 512, 1040, 9, gated=gated), act, keep_z=True)


@pytest.mark.parametrize("knobs", [{"cluster": 0}, {"cluster_size": 8}, {"max_ctas": 2}, {"max_token_tile": 64},
                                   {"pair_mma": 0}, {"widen_min_m": 129}, {"pdl": 0}, {"pair_split": 1},
                                   {"convert_max_m": 4096}])
@pytest.mark.parametrize("fmt", FMTS)
def test_forward_modes(q, oracle, fmt, knobs):
    with q.knobs(**knobs):
        for M in (16, 150, 600):
            for gated in (False, True):
                check_forward(Layer(q, oracle, fmt, M, 640, 1168, 12, gated=gated), "silu", keep_z=True)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [96, 97, 129, 200, 256, 257])
@pytest.mark.parametrize("knobs", [{}, {"widen_min_m": 0}, {"pair_mma": 0}], ids=str)
def test_first_pair_tile(q, oracle, fmt, M, knobs):
    """INT4 converted inside the kernel or widened, one CTA or pairs."""
    with q.knobs(**knobs):
        check_forward(Layer(q, oracle, fmt, M, 512, 400, 21), "silu", keep_z=True)
        check_forward(Layer(q, oracle, fmt, M, 512, 400, 0, gated=True), "gelu_tanh")


@pytest.mark.parametrize("fmt", FMTS)
def test_first_pair_tile_of_a_large_layer(q, oracle, fmt):
    """Too many weights to widen at this token count."""
    check_forward(Layer(q, oracle, fmt, 130, 4096, 4352, 9), "relu")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 16, 50, 100, 600])
def test_plain_epilogue_equals_forward(q, oracle, fmt, M):
    """Without bias, activation and residual: qlin_forward, bit for bit; Z too."""
    L = Layer(q, oracle, fmt, M, 768, 528, 17, bias=False, residual=False)
    Z = torch.empty((M, 528), dtype=torch.float16, device="cuda")
    Y, _ = L.forward("none", Z=Z)
    Yf = torch.empty_like(Y)
    n = q.qlin_forward_workspace(M, L.w)
    q.qlin_forward(L.dX, M, L.w, cuda(L.s), GAMMA, False, Yf, q.empty_workspace(n), n)
    assert torch.equal(Y, Yf) and torch.equal(Z, Yf)


@pytest.mark.parametrize("M", [3, 90, 513])
def test_residual_in_place(q, oracle, M):
    L = Layer(q, oracle, synth.W4_PERCHANNEL, M, 512, 656, 9)
    want, _ = L.forward("gelu")
    Y = cuda(L.res)
    got, _ = L.forward("gelu", Y=Y, res=Y)
    assert torch.equal(want, got)


@pytest.mark.parametrize("nO", [0, 9])
@pytest.mark.parametrize("N", [16, 80, 144, 272, 2064])
def test_many_tiles_with_residual(q, oracle, N, nO):
    """Several tiles per pair of CTAs, ragged at both ends, with and without
    the kept pre-activation; the residual replaced in place."""
    for M in (400, 2600 if N < 2000 else 2900):
        L = Layer(q, oracle, synth.W8_PERCHANNEL, M, 128, N, nO)
        want = check_forward(L, "silu", keep_z=True)
        assert torch.equal(want, check_forward(L, "silu"))
        Y = cuda(L.res)
        assert torch.equal(want, L.forward("silu", Y=Y, res=Y)[0])
        check_forward(Layer(q, oracle, synth.W8_PERCHANNEL, M, 128, N, nO, gated=True), "gelu", keep_z=True)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("nO", [0, 13])
@pytest.mark.parametrize("M,N", [(1500, 2064), (2300, 2320), (2900, 1808)])
def test_whole_and_half_tiles(q, oracle, fmt, nO, M, N):
    """Fewer tiles than pairs of CTAs, but more than half of them; one wave and
    a few, a wave and a half: whole tiles alone and before half tiles, with an
    odd number of 128-channel blocks."""
    check_forward(Layer(q, oracle, fmt, M, 256, N, nO), "gelu", keep_z=True)
    check_forward(Layer(q, oracle, fmt, M, 256, N, nO, gated=True), "silu")


def test_rows_and_columns_outside_are_left(q, oracle):
    """Nothing behind the last token or the last channel's row is written."""
    for M in (1, 17, 70, 300):
        for gated in (False, True):
            L = Layer(q, oracle, synth.W8_PERCHANNEL, M, 256, 272, 4, gated=gated)
            Y = torch.full((M + 3, L.Nout), 7.0, dtype=torch.float16, device="cuda")
            Z = torch.full((M + 3, L.N), 7.0, dtype=torch.float16, device="cuda")
            L.forward("silu", Y=Y, Z=Z)
            assert (Y[M:] == 7).all() and (Z[M:] == 7).all()


def test_extreme_preactivations(q, oracle):
    """Pre-activations up to fp16's ends: no NaN, the limits 0 and z."""
    for M in (2, 300):
        L = Layer(q, oracle, synth.W8_PERCHANNEL, M, 128, 64, 0, residual=False)
        L.bias = np.where(np.arange(64) % 2 == 0, 60000, -60000).astype(np.float32)
        L.dXb = cuda(L.bias)
        for act in ref.ACTS[1:]:
            check_forward(L, act)
            y = host(L.forward(act)[0])
            assert np.all(y[:, 1::2] == 0) and np.all(y[:, 0::2] > 59000)


def test_zero_tokens_and_zero_rows(q, oracle):
    L = Layer(q, oracle, synth.W8_PERCHANNEL, 4, 128, 64, 3)
    L.X[2] = 0
    L.dX = cuda(L.X)
    check_forward(L, "gelu", keep_z=True)
    q.qlin_forward_act(None, 0, L.w, None, GAMMA, True, None, None, 0)
    q.qlin_forward_gated(None, 0, L.w, None, GAMMA, True, None, None, 0)
    db = torch.ones(64, device="cuda")
    q.qlin_backward_act(L.w, None, None, 0, None, None, db, None, 0)
    assert (db == 0).all()


def test_pack_gated_equals_interleaved(q, oracle):
    for fmt in FMTS:
        L = Layer(q, oracle, fmt, 1, 256, 304, 11, gated=True)
        other = q.PackedLayer.pack(cuda(L.W), L.O, fmt)
        assert torch.equal(L.layer.buffer, other.buffer)


# ---------------------------------------------------------------- backward

def check_backward(L, act, seed=1, dy_std=2.0 ** -7, with_dbias=True, z=None):
    q, rng = L.q, np.random.default_rng(seed)
    Z = rng.standard_normal((L.M, L.N)).astype(np.float16) * np.float16(1.5) if z is None else z
    dY = (rng.standard_normal((L.M, L.Nout)) * dy_std).astype(np.float16)
    Zd, dYd, sd = cuda(Z), cuda(dY), cuda(L.s)
    dX = torch.full((L.M, L.K), float("nan"), dtype=torch.float16, device="cuda")
    db = torch.full((L.N,), float("nan"), device="cuda") if with_dbias else None
    size = q.qlin_backward_gated_workspace if L.gated else q.qlin_backward_act_workspace
    ws, n = ws_for(q, size(L.M, L.w))
    ws.fill_(255)  # no zero-fill needed
    call = q.qlin_backward_gated if L.gated else q.qlin_backward_act
    got = []
    for _ in range(2):
        call(L.w, dYd, Zd, L.M, sd, dX, db, ws, n, act=ref.ACTS.index(act))
        got.append((dX.clone(), None if db is None else db.clone()))
    q.qlin_poll_device_status()
    assert torch.equal(got[0][0], got[1][0])
    z, dy = Z.astype(np.float64), dY.astype(np.float64)
    dz, err = ref.dz_gated(dy, z, act) if L.gated else ref.dz_act(dy, z, act)
    if L.gated:
        top = (np.abs(dy) * np.maximum(np.abs(z[:, 0::2]), np.abs(z[:, 1::2]))).max(1)
    else:
        top = np.abs(dy).max(1)
    want, bound = ref.input_gradient(dz, err, top, L.pk, L.W, L.s)
    within(host(got[0][0]), want, bound, "dX")
    if with_dbias:
        assert torch.equal(got[0][1], got[1][1])
        want, bound = ref.bias_gradient(dz, err)
        within(host(got[0][1]), want, bound + 2.0 ** -120, "dbias")


BWD_SHAPES = [(1, 512, 256, 10), (19, 96, 48, 0), (131, 1056, 1040, 21), (256, 640, 272, 64), (600, 384, 1168, 300)]


@pytest.mark.parametrize("i,shape", list(enumerate(BWD_SHAPES)))
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("gated", [False, True])
def test_backward(q, oracle, fmt, gated, i, shape):
    M, K, N, nO = shape
    K = -(-K // 128) * 128 if fmt == synth.W4_G128 else K
    L = Layer(q, oracle, fmt, M, K, N, nO, gated=gated)
    check_backward(L, ref.ACTS[(i + fmt) % 5], with_dbias=i % 2 == 0)


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("gated", [False, True])
def test_backward_every_activation(q, oracle, act, gated):
    check_backward(Layer(q, oracle, synth.W8_PERCHANNEL, 70, 256, 528, 12, gated=gated), act)


@pytest.mark.parametrize("N", [1040, 4112, 8208, 12304, 16400, 24592, 32768, 32784, 40000])
@pytest.mark.parametrize("gated", [False, True])
def test_backward_wide_layers(q, oracle, gated, N):
    """Every width class of the activation's backward pass, on both sides of
    its edges and past the last."""
    for M, with_dbias in ((3, True), (310, True), (5, False)):
        check_backward(Layer(q, oracle, synth.W8_PERCHANNEL, M, 128, N, 2, gated=gated), "silu", with_dbias=with_dbias)
    check_backward(Layer(q, oracle, synth.W8_PERCHANNEL, 4, 128, N, 2, gated=gated), "none")


@pytest.mark.parametrize("dy_std", [3e-7, 2.0 ** -7, 3000.0])
def test_backward_gradient_scales(q, oracle, dy_std):
    """The row's power of two keeps tiny and huge gradients in range: dH * up
    alone would leave fp16 at the large end and lose its digits at the small."""
    L = Layer(q, oracle, synth.W8_PERCHANNEL, 33, 256, 512, 6, gated=True)
    rng = np.random.default_rng(5)
    z = rng.standard_normal((33, 512))
    z[:, 1::2] *= 30 if dy_std > 1 else 1
    check_backward(L, "silu", dy_std=dy_std, z=z.astype(np.float16))


def test_backward_one_output_only(q, oracle):
    L = Layer(q, oracle, synth.W4_PERCHANNEL, 40, 256, 272, 8)
    n = q.qlin_backward_act_workspace(40, L.w)
    ws = q.empty_workspace(n)
    Z, dY = cuda(L.res), cuda(L.res[::-1].copy())
    both = torch.empty(40, 256, dtype=torch.float16, device="cuda"), torch.empty(272, device="cuda")
    one = torch.empty_like(both[0]), torch.empty_like(both[1])
    q.qlin_backward_act(L.w, dY, Z, 40, cuda(L.s), *both, ws, n, act=4)
    q.qlin_backward_act(L.w, dY, Z, 40, cuda(L.s), one[0], None, ws, n, act=4)
    q.qlin_backward_act(L.w, dY, Z, 40, None, None, one[1], ws, n, act=4)
    assert torch.equal(both[0], one[0]) and torch.equal(both[1], one[1])


def test_backward_infinite_gradient_shows(q, oracle):
    """An infinity in one token's gradient reaches that token's dX (a loss
    scaler looks for it) and no other token's."""
    L = Layer(q, oracle, synth.W8_PERCHANNEL, 12, 128, 256, 0)
    dY = np.full((12, 256), 2.0 ** -7, np.float16)
    dY[3, 100] = np.inf
    dY[5, 17] = np.nan
    n = q.qlin_backward_act_workspace(12, L.w)
    dX = torch.empty(12, 128, dtype=torch.float16, device="cuda")
    q.qlin_backward_act(L.w, cuda(dY), None, 12, None, dX, None, q.empty_workspace(n), n)
    bad = ~np.isfinite(host(dX).astype(np.float32)).all(1)
    assert bad[3] and bad[5] and bad.sum() == 2


# ---------------------------------------------------------------- streams, graphs

def test_graph_replay_and_streams(q, oracle):
    """Forward and backward captured once and replayed on new inputs; two
    streams with their own workspaces at once."""
    L = Layer(q, oracle, synth.W4_G128, 40, 512, 528, 9, gated=True)
    s, sd = cuda(L.s), cuda(L.s)
    Y = torch.empty(40, 264, dtype=torch.float16, device="cuda")
    Z = torch.empty(40, 528, dtype=torch.float16, device="cuda")
    dX = torch.empty(40, 512, dtype=torch.float16, device="cuda")
    db = torch.empty(528, device="cuda")
    n = q.qlin_backward_gated_workspace(40, L.w)
    ws = q.empty_workspace(n)

    def step():
        L.forward("silu", update=True, Z=Z, s=s, Y=Y)
        q.qlin_backward_gated(L.w, Y, Z, 40, s, dX, db, ws, n)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in range(3):
        x = torch.randn(40, 512, device="cuda").half()
        L.dX.copy_(x)
        s.copy_(sd)
        g.replay()
        got = [t.clone() for t in (Y, Z, dX, db, s)]
        s.copy_(sd)
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (Y, Z, dX, db, s)):
            assert torch.equal(a, b), k
    A = Layer(q, oracle, synth.W8_PERCHANNEL, 600, 512, 528, 9)
    B = Layer(q, oracle, synth.W8_PERCHANNEL, 16, 512, 528, 9, gated=True)
    want = A.forward("gelu")[0], B.forward("silu")[0]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    sa, sb, ra = cuda(A.s), cuda(B.s), cuda(A.res)
    outs = [(torch.empty_like(want[0]), torch.empty_like(want[1])) for _ in range(8)]
    torch.cuda.synchronize()
    for ya, yb in outs:
        A.forward("gelu", s=sa, Y=ya, res=ra, stream=st[0])
        B.forward("silu", s=sb, Y=yb, stream=st[1])
    torch.cuda.synchronize()
    for ya, yb in outs:
        assert torch.equal(ya, want[0]) and torch.equal(yb, want[1])


# ---------------------------------------------------------------- refusals (binding)

def test_binding_refuses(q, oracle):
    L = Layer(q, oracle, synth.W8_PERCHANNEL, 8, 128, 64, 3)
    for bad in (L.dX.float(), L.dX.t(), L.dX[:4], L.dX.cpu()):
        good, L.dX = L.dX, bad
        with pytest.raises(ValueError):
            L.forward("none")
        L.dX = good
    with pytest.raises(ValueError):
        L.forward("none", Z=torch.empty(8, 63, dtype=torch.float16, device="cuda"))
