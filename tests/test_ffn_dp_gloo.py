"""Data-parallel host logic of the feed-forward block on CPU: two gloo ranks
combine their column maxima by `max_over_ranks`, in the block's own order of
calls, a rank without tokens among them.  The library's calls are stood in for
by numpy (there is no GPU here)."""
import datetime

import numpy as np
import pytest
import torch
import torch.multiprocessing as mp

from test_dp_gloo import _free_port


class FakeLayer:
    def __init__(self, K, N, O, seed):
        rng = np.random.default_rng(seed)
        self.K, self.N, self.O, self.n_outlier = K, N, O, len(O)
        self.W = rng.standard_normal((K, N)).astype(np.float32) * 0.1
        self.wmax = np.abs(self.W[O]).max(1) if len(O) else np.zeros(0, np.float32)
        self.buffer = torch.zeros(1)
        self.w = self


def fake(qlin, log):
    """Stand-ins: a layer's input is divided by its scales at the outliers, so
    each stage depends on the state before it."""
    def size(*a):
        return 0

    def norm(X, M, K, kind, gamma, beta, eps, Y, mean, rstd, stream=None):
        Y.copy_(X)
        if rstd is not None:
            rstd.fill_(1)

    def colmax(x, M, w, cmax, stream=None):
        cmax.zero_()
        if M:
            cmax.copy_(x[:, torch.from_numpy(w.O).long()].float().abs().amax(0))

    def momentum(w, cmax, s, gamma, stream=None):
        beta = np.maximum(1, np.sqrt(cmax.numpy() / w.wmax))
        s.copy_(torch.from_numpy((gamma * s.numpy() + (1 - gamma) * beta).astype(np.float32)))

    def layer(x, w, s):
        x = x.float().clone()
        x[:, torch.from_numpy(w.O).long()] /= s
        W = torch.from_numpy(w.W)
        # row by row: the same operations whatever rows are beside it
        return torch.stack([(r[:, None] * W).sum(0) for r in x]) if len(x) else x.new_empty(0, w.N)

    def gated(X, M, w, s, gamma, update, H, ws, n, act=4, bias=None, Z=None, stream=None):
        log.append(("gated", update))
        z = layer(X, w, s)
        H.copy_(z[:, 0::2] * z[:, 1::2])

    def act(X, M, w, s, gamma, update, Y, ws, n, act=0, bias=None, residual=None, Z=None, stream=None):
        log.append(("down", update))
        Y.copy_(layer(X, w, s) + residual.float())

    for name in ("forward_gated", "forward_act", "backward_gated", "backward_act", "norm_backward"):
        setattr(qlin, f"qlin_{name}_workspace", size)
    qlin.qlin_norm_forward, qlin.qlin_outlier_colmax, qlin.qlin_momentum_update = norm, colmax, momentum
    qlin.qlin_forward_gated, qlin.qlin_forward_act = gated, act


def block(reduce_max, log):
    from quantized_linear_layers_token_b200 import ffn, qlin
    fake(qlin, log)
    torch.cuda.is_current_stream_capturing = lambda: False
    D, F = 32, 48
    gated = FakeLayer(D, 2 * F, np.array([1, 7, 30], np.int32), 1)
    down = FakeLayer(F, D, np.array([0, 5], np.int32), 2)
    return ffn.GatedFeedForward(gated, down, torch.ones(D), reduce_max=reduce_max)


def shards():
    x = torch.from_numpy(np.random.default_rng(3).standard_normal((10, 32)).astype(np.float16))
    return [[x[:3], x[3:]], [x[:0], x]]  # uneven, and a rank without tokens


def _worker(rank, world, port, q):
    import torch.distributed as dist
    dist.init_process_group("gloo", init_method=f"tcp://127.0.0.1:{port}", rank=rank, world_size=world,
                            timeout=datetime.timedelta(seconds=60))
    try:
        from quantized_linear_layers_token_b200.dp import max_over_ranks
        out = []
        for parts in shards():
            log = []
            b = block(max_over_ranks(), log)
            for _ in range(2):
                y, saved = b.forward(parts[rank], training=True)
            out.append((y.numpy().copy(), saved.s_gated.numpy().copy(), saved.s_down.numpy().copy(), log))
        q.put((rank, out))
    finally:
        dist.destroy_process_group()


def _single(q):
    out = []
    for parts in shards():
        b = block(lambda t: None, [])
        for _ in range(2):
            y, saved = b.forward(torch.cat(parts), training=True)
        out.append((y.numpy().copy(), saved.s_gated.numpy().copy(), saved.s_down.numpy().copy()))
    q.put((-1, out))


@pytest.mark.timeout(300)
def test_two_ranks_keep_one_state():
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    port = _free_port()
    procs = [ctx.Process(target=_worker, args=(r, 2, port, q)) for r in range(2)] + [ctx.Process(target=_single, args=(q,))]
    for p in procs:
        p.start()
    got = dict(q.get(timeout=120) for _ in procs)
    for p in procs:
        p.join(timeout=60)
        assert p.exitcode == 0
    for k in range(2):
        a, b, whole = got[0][k], got[1][k], got[-1][k]
        assert a[3] == b[3] == [("gated", False), ("down", False)] * 2  # the layers' calls leave the states alone
        for i in (1, 2):
            np.testing.assert_array_equal(a[i], b[i])
            np.testing.assert_array_equal(a[i], whole[i])
        np.testing.assert_array_equal(np.concatenate([a[0], b[0]]), whole[0])


def test_max_over_ranks_alone():
    """Without a process group, or in one of a single rank: the rank's own maxima."""
    from quantized_linear_layers_token_b200.dp import max_over_ranks
    t = torch.tensor([1.0, 2.0])
    max_over_ranks()(t)
    assert t.tolist() == [1.0, 2.0]
