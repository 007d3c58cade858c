"""Data-parallel training forward of the feed-forward block: two replicas with
their own tokens, whose column maxima are combined on the host, keep one state,
that of the update over all tokens.  The replicas' kernels do not wait for one
another."""
import threading

import numpy as np
import pytest
import torch

from quantized_linear_layers_token_b200 import synth
from test_gpu_ffn import Block, h16, q  # noqa: F401 (q: fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 40, 300])
def test_one_replica_alone(q, oracle, M):  # noqa: F811
    """With nothing to combine: the bits of the update inside the layers' calls."""
    args = (q, oracle, synth.W4_PERCHANNEL, 256, 384, 7, q.QLIN_NORM_RMS, False)
    a, b = Block(*args), Block(*args)
    b.ffn.reduce_max = lambda t: None
    x = a.c(a.x(M, 256))
    for _ in range(2):
        (ya, sa), (yb, sb) = a.ffn.forward(x, training=True), b.ffn.forward(x, training=True)
        assert torch.equal(ya, yb) and torch.equal(sa.z, sb.z)
        assert torch.equal(sa.s_gated, sb.s_gated) and torch.equal(sa.s_down, sb.s_down)
    s = b.ffn.s_gated.clone()
    b.ffn.forward(x)  # serving leaves the state
    assert torch.equal(s, b.ffn.s_gated)
    q.qlin_poll_device_status()


@pytest.mark.parametrize("counts", [(5, 40), (200, 1), (0, 33)], ids=str)
def test_two_replicas(q, oracle, counts):  # noqa: F811
    D, F = 256, 384
    blocks = [Block(q, oracle, synth.W8_PERCHANNEL, D, F, 7, q.QLIN_NORM_RMS, False) for _ in counts]
    xs = [blocks[0].c(blocks[0].x(max(M, 1), D)[:M]) for M in counts]
    barrier, slots = threading.Barrier(2, timeout=60), [None, None]
    results, errors = [None, None], []

    def reduce_for(r):
        def reduce(t):  # the host exchanges; no kernel of one replica waits for the other's
            slots[r] = t.cpu()
            barrier.wait()
            top = torch.maximum(*slots)
            barrier.wait()
            t.copy_(top)
        return reduce

    def replica(r):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                b = blocks[r].ffn
                b.reduce_max = reduce_for(r)
                for _ in range(2):
                    y, saved = b.forward(xs[r], training=True)
                stream.synchronize()
                results[r] = y, saved
        except Exception as e:  # noqa: BLE001 (shown by the test)
            errors.append(e)
            barrier.abort()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=replica, args=(r,)) for r in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    q.qlin_poll_device_status()
    a, b = results[0][1], results[1][1]
    assert torch.equal(a.s_gated, b.s_gated) and torch.equal(a.s_down, b.s_down)
    # the gated layer's state is the oracle's over all tokens (its input does not depend on any scale)
    L = blocks[0]
    x = torch.cat(xs)
    n = torch.empty_like(x)
    q.qlin_norm_forward(x, x.shape[0], D, q.QLIN_NORM_RMS, L.ffn.gamma, None, L.ffn.eps, n)
    s = np.ones(7, np.float32)
    for _ in range(2):
        s = L.oracle.momentum_update(h16(n), L.Og, L.pg["wmaxO"], 0.9, s)
    assert np.array_equal(a.s_gated.cpu().numpy(), s)
    # ... and a replica by itself has another
    alone = Block(q, oracle, synth.W8_PERCHANNEL, D, F, 7, q.QLIN_NORM_RMS, False)
    alone.ffn.forward(xs[int(np.argmin(counts))], training=True)
    assert not torch.equal(alone.ffn.s_gated, a.s_gated)
