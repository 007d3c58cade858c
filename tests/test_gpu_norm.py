"""GPU parity of the layer norm and the RMS norm, forward and backward,
against 64-bit references (fused_ref.py)."""
import numpy as np
import pytest
import torch

import fused_ref as ref

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_linear_layers_token_b200 import qlin
    qlin.lib()
    return qlin


def cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def nan(*shape, dtype=torch.float32):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def within(got, want, bound, what):
    got = got.double().cpu().numpy()
    assert np.all(np.isfinite(got)), what
    over = np.abs(got - want) / bound
    assert np.all(over <= 1), (what, float(over.max()))


def draw(M, K, offset=0.3, seed=0):
    rng = np.random.default_rng([seed, M, K])
    x = rng.standard_normal((M, K)) + offset
    x[:, rng.choice(K, max(1, K // 100), replace=False)] *= 40
    gamma = (1 + 0.1 * rng.standard_normal(K)).astype(np.float32)
    beta = (0.1 * rng.standard_normal(K)).astype(np.float32)
    dy = (rng.standard_normal((M, K)) / 128).astype(np.float16)
    dres = (rng.standard_normal((M, K)) / 128).astype(np.float16)
    return x.astype(np.float16), gamma, beta, dy, dres


def forward(q, x, gamma, beta, rms, eps=EPS):
    M, K = x.shape
    Y, mean, rstd = nan(M, K, dtype=torch.float16), nan(M), nan(M)
    q.qlin_norm_forward(cuda(x), M, K, int(rms), cuda(gamma), cuda(beta), eps, Y, mean, rstd)
    return Y, mean, rstd


def check(q, x, gamma, beta, dy, dres, rms, eps=EPS):
    M, K = x.shape
    Y, mean, rstd = forward(q, x, gamma, beta, rms, eps)
    y, yb, mu, r, mub, rb = ref.norm_forward(x, gamma, beta, np.float32(eps), rms)
    within(Y, y, yb, "Y")
    within(rstd, r, rb + 2.0 ** -22 * r, "rstd")
    if rms:
        assert torch.isnan(mean).all()  # not written
        mean = None
    else:
        within(mean, mu, mub + 2.0 ** -23 * np.abs(mu) + 1e-30, "mean")
    n = q.qlin_norm_backward_workspace(M, K)
    ws = q.empty_workspace(n)
    ws.fill_(255)  # no zero-fill needed
    dX, dg, db = nan(M, K, dtype=torch.float16), nan(K), nan(K)
    args = (cuda(dy), cuda(x), M, K, int(rms), cuda(gamma), mean, rstd, cuda(dres))
    q.qlin_norm_backward(*args, dX, dg, db, ws, n)
    want = ref.norm_backward(dy, x, gamma, None if rms else mean.cpu().numpy(), rstd.cpu().numpy(), dres, rms)
    within(dX, want[0], want[1], "dX")
    within(dg, want[2], want[3] + 1e-30, "dgamma")
    within(db, want[4], want[5] + 1e-30, "dbeta")
    again = nan(M, K, dtype=torch.float16), nan(K), nan(K)
    q.qlin_norm_backward(*args, *again, ws, n)
    for a, b in zip((dX, dg, db), again):
        assert torch.equal(a, b)


# a vector short of a warp, one warp, odd multiples of 32, each row width class and its edges, the largest
KS = [32, 96, 256, 288, 1024, 1056, 2048, 4096, 4128, 8192, 8224, 16384, 16416, 32768, 65536]


@pytest.mark.parametrize("K", KS)
@pytest.mark.parametrize("rms", [False, True])
def test_widths(q, K, rms):
    x, gamma, beta, dy, dres = draw(5, K)
    check(q, x, gamma, beta, dy, dres, rms)
    check(q, x, gamma, None, dy, None, rms)


@pytest.mark.parametrize("M", [1, 2, 3, 7, 147, 149, 1000, 2501])
@pytest.mark.parametrize("rms", [False, True])
def test_token_counts(q, M, rms):
    for K in (64, 1056, 4096):
        check(q, *draw(M, K), rms)


def test_many_short_rows(q):
    check(q, *draw(70001, 32), False)


def test_large_mean(q):
    """A mean a thousand times the spread: the squares are summed after it
    is subtracted."""
    x, gamma, beta, dy, dres = draw(9, 2048, offset=1000.0)
    check(q, x, gamma, beta, dy, dres, False)


def test_constant_and_zero_rows(q):
    x, gamma, beta, dy, dres = draw(6, 512)
    x[1] = 0
    x[4] = 3.5
    for rms in (False, True):
        check(q, x, gamma, beta, dy, dres, rms)
    Y, _, rstd = forward(q, x, gamma, beta, False)
    assert torch.equal(Y[4], cuda(beta).half()) and abs(rstd[1].item() - EPS ** -0.5) < 1e-3


def test_extreme_values(q):
    x, gamma, beta, dy, dres = draw(4, 1024)
    x[0] = 65504
    x[0, ::2] = -65504
    x[1] = np.float16(6e-8)
    check(q, x, gamma, beta, dy, dres, False)
    check(q, x, gamma, beta, dy, dres, True)


def test_infinite_rows_stay_in_their_rows(q):
    x, gamma, beta, _, _ = draw(6, 256)
    clean, _, _ = forward(q, x, gamma, beta, False)
    x[2, 17] = np.inf
    x[4, 3] = np.nan
    Y, _, _ = forward(q, x, gamma, beta, False)
    bad = ~torch.isfinite(Y).all(1)
    assert bad.tolist() == [False, False, True, False, True, False]
    assert torch.equal(Y[~bad], clean[~bad])


@pytest.mark.parametrize("K", [96, 4096, 8224, 32768])
@pytest.mark.parametrize("alias", ["dY", "X", "dres"])
def test_in_place(q, K, alias):
    x, gamma, beta, dy, dres = draw(300, K)
    Y, mean, rstd = forward(q, x, gamma, beta, False)
    xd = cuda(x)
    q.qlin_norm_forward(xd, 300, K, 0, cuda(gamma), cuda(beta), EPS, xd)
    assert torch.equal(xd, Y)
    n = q.qlin_norm_backward_workspace(300, K)
    out = []
    for own in (True, False):
        t = {"dY": cuda(dy), "X": cuda(x), "dres": cuda(dres)}
        dX = nan(300, K, dtype=torch.float16) if own else t[alias]
        dg, db = nan(K), nan(K)
        q.qlin_norm_backward(t["dY"], t["X"], 300, K, 0, cuda(gamma), mean, rstd, t["dres"], dX, dg, db,
                             q.empty_workspace(n), n)
        out.append((dX, dg, db))
    for a, b in zip(*out):
        assert torch.equal(a, b)


@pytest.mark.parametrize("K", [256, 4096, 32768])
def test_wanted_outputs_only(q, K):
    x, gamma, beta, dy, dres = draw(40, K)
    _, mean, rstd = forward(q, x, gamma, beta, False)
    n = q.qlin_norm_backward_workspace(40, K)
    ws = q.empty_workspace(n)
    base = (cuda(dy), cuda(x), 40, K, 0, cuda(gamma), mean, rstd, cuda(dres))
    full = nan(40, K, dtype=torch.float16), nan(K), nan(K)
    q.qlin_norm_backward(*base, *full, ws, n)
    dX = torch.empty_like(full[0])
    q.qlin_norm_backward(*base, dX, None, None)  # no workspace needed
    assert torch.equal(dX, full[0])
    for k in (1, 2):
        out = [None, None, None]
        out[k] = nan(K)
        q.qlin_norm_backward(*base, *out, ws, n)
        assert torch.equal(out[k], full[k])


def test_no_rows(q):
    dg, db = nan(64), nan(64)
    q.qlin_norm_forward(None, 0, 64, 0, None, None, EPS, None)
    q.qlin_norm_backward(None, None, 0, 64, 0, None, None, None, None, None, dg, db)
    assert (dg == 0).all() and (db == 0).all()
    assert q.qlin_norm_backward_workspace(0, 64) == 0


def test_rows_behind_the_last_are_left(q):
    for K in (64, 1024, 4096, 16416):
        x, gamma, beta, dy, dres = draw(5, K)
        Y = torch.full((7, K), 9.0, dtype=torch.float16, device="cuda")
        mean, rstd = torch.full((7,), 9.0, device="cuda"), torch.full((7,), 9.0, device="cuda")
        q.qlin_norm_forward(cuda(x), 5, K, 0, cuda(gamma), None, EPS, Y, mean, rstd)
        dX = torch.full((7, K), 9.0, dtype=torch.float16, device="cuda")
        q.qlin_norm_backward(cuda(dy), cuda(x), 5, K, 0, cuda(gamma), mean, rstd, None, dX, None, None)
        for t in (Y, mean, rstd, dX):
            assert (t[5:] == 9).all() and not (t[:5] == 9).all()


def test_graph_replay(q):
    x, gamma, beta, dy, dres = draw(200, 4096)
    X, g, b, D, R = (cuda(t) for t in (x, gamma, beta, dy, dres))
    Y, mean, rstd = nan(200, 4096, dtype=torch.float16), nan(200), nan(200)
    dX, dg, db = nan(200, 4096, dtype=torch.float16), nan(4096), nan(4096)
    n = q.qlin_norm_backward_workspace(200, 4096)
    ws = q.empty_workspace(n)

    def step():
        q.qlin_norm_forward(X, 200, 4096, 0, g, b, EPS, Y, mean, rstd)
        q.qlin_norm_backward(D, X, 200, 4096, 0, g, mean, rstd, R, dX, dg, db, ws, n)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        X.copy_(torch.randn(200, 4096, device="cuda"))
        graph.replay()
        got = [t.clone() for t in (Y, dX, dg, db)]
        step()
        torch.cuda.synchronize()
        for a, c in zip(got, (Y, dX, dg, db)):
            assert torch.equal(a, c)
