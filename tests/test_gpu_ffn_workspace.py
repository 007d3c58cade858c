"""The feed-forward block's workspace: shared by the blocks of a model, grown
by token counts and captures in any order, and made ready again after a
bounded wait gave up.  Every result is that of a block of its own."""
import pytest
import torch

from quantized_linear_layers_token_b200 import synth
from test_gpu_ffn import Block, q  # noqa: F401 (q: fixture)

pytestmark = pytest.mark.gpu


def step(block, x, dy):
    """A training step from given momentum states, which it leaves as they were."""
    keep = block.s_gated.clone(), block.s_down.clone()
    y, saved = block.forward(x, training=True)
    g = block.backward(saved, dy)
    out = [y, saved.s_gated, saved.s_down, *(g[k] for k in sorted(g) if g[k] is not None)]
    block.s_gated.copy_(keep[0])
    block.s_down.copy_(keep[1])
    return out


def equal(a, b):
    return len(a) == len(b) and all(torch.equal(s, t) for s, t in zip(a, b))


def test_blocks_of_a_model_share_one(q, oracle):  # noqa: F811
    from quantized_linear_layers_token_b200.ffn import Workspace
    shapes = [(synth.W4_G128, 512, 640, 9), (synth.W8_PERCHANNEL, 256, 1408, 30), (synth.W4_PERCHANNEL, 768, 384, 0)]
    own = [Block(q, oracle, *s, q.QLIN_NORM_LAYER, bias=True) for s in shapes]
    ws = Workspace()
    blocks = [Block(q, oracle, *s, q.QLIN_NORM_LAYER, bias=True) for s in shapes]
    for b in blocks:
        b.ffn.workspace = ws
    xs = {(i, M): b.c(b.x(M, s[1])) for i, (b, s) in enumerate(zip(own, shapes)) for M in (1, 20, 100, 300, 600)}
    for M in (20, 600, 1, 300, 100, 20, 300):
        for i, b in enumerate(blocks):
            x = xs[i, M]
            assert equal(step(b.ffn, x, x), step(own[i].ffn, x, x)), (i, M)
            assert torch.equal(b.ffn.forward(x), own[i].ffn.forward(x)), (i, M)
    assert ws._buf.numel() == max(b.ffn.workspace_bytes(600, training=True) for b in blocks)
    q.qlin_poll_device_status()


def test_captures_around_a_growing_buffer(q, oracle):  # noqa: F811
    """Graphs captured on the buffer, on the one after it and without one that
    is large enough, replayed in turn with eager calls."""
    b = Block(q, oracle, synth.W4_G128, 256, 384, 5, q.QLIN_NORM_RMS, bias=False)
    own = Block(q, oracle, synth.W4_G128, 256, 384, 5, q.QLIN_NORM_RMS, bias=False)
    graphs = []

    def capture(M):
        x = b.c(b.x(M, 256))
        dy = torch.randn(M, 256, device="cuda").half() / 128
        want = step(own.ffn, x, dy)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(b.ffn, x, dy)
        graphs.append((g, out, want, x, dy))  # (the graph reads x and dy)

    b.ffn.workspace.reserve(b.ffn.workspace_bytes(40, training=True))
    capture(40)
    capture(300)                       # too large for the buffer
    x = b.c(b.x(600, 256))
    small = b.ffn.workspace._buf.numel()
    step(b.ffn, x, x)                  # grows it: the first graph keeps the old one
    assert b.ffn.workspace._buf.numel() > small
    capture(300)
    assert len(b.ffn.workspace._captured) == 2
    junk = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(64)]
    for k in (2, 0, 1, 0, 2, 1, 1):
        g, out, want = graphs[k][:3]
        for t in out:
            t.zero_()
        g.replay()
        assert equal(out, want), k
        assert torch.equal(b.ffn.forward(x), own.ffn.forward(x))
    del junk
    q.qlin_poll_device_status()


def test_reset_after_a_wait_gave_up(q, oracle):  # noqa: F811
    """Waits without time give up; after reset() every token count is right
    again, eagerly and in a graph captured before, whatever the workspace holds."""
    D, F = 16384, 1024
    gen = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda").half()  # noqa: E731
    import numpy as np
    from quantized_linear_layers_token_b200.ffn import GatedFeedForward
    O = np.arange(9, dtype=np.int32) * 5
    gated = q.PackedLayer.pack_gated(n(D, F) * 0.02, n(D, F) * 0.02, O, synth.W8_PERCHANNEL)
    down = q.PackedLayer.pack(n(F, D) * 0.02, O, synth.W8_PERCHANNEL)
    gamma = torch.ones(D, device="cuda")
    make = lambda: GatedFeedForward(gated, down, gamma)  # noqa: E731
    block = make()
    xs = {M: n(M, D) for M in (1, 16, 40, 90, 300, 600)}
    want = {M: step(make(), x, x) for M, x in xs.items()}
    q.qlin_poll_device_status()
    block.workspace.reserve(block.workspace_bytes(600, training=True))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(block, xs[16], xs[16])
    keep = block.s_gated.clone(), block.s_down.clone()
    with q.knobs(wait_ns=0):
        block.forward(xs[600], training=True)
        with pytest.raises(q.QlinError) as e:
            q.qlin_poll_device_status()
        assert q.STATUS[e.value.status] == "QLIN_ERR_TIMEOUT"
    block.s_gated.copy_(keep[0])
    block.s_down.copy_(keep[1])
    block.workspace.get(1).fill_(255)  # whatever state such a call may leave
    block.reset()
    for M in (600, 16, 1, 300, 90, 40):
        assert equal(step(block, xs[M], xs[M]), want[M]), M
    graph.replay()
    assert equal(out, want[16])
    q.qlin_poll_device_status()


def test_memory_of_a_large_block(q):  # noqa: F811
    """A training step's workspace is the largest call's, not the calls' sum,
    and a second block adds nothing."""
    from quantized_linear_layers_token_b200.ffn import GatedFeedForward, Workspace
    ws = Workspace()
    D, F, M = 2048, 5632, 1024
    blocks = []
    for _ in range(2):
        gated = q.PackedLayer(D, 2 * F, synth.W4_G128, 0)
        down = q.PackedLayer(F, D, synth.W4_G128, 0)
        blocks.append(GatedFeedForward(gated, down, torch.ones(D, device="cuda"), workspace=ws))
    x = torch.zeros(M, D, dtype=torch.float16, device="cuda")
    used = []
    for b in blocks:
        y, saved = b.forward(x, training=True)
        b.backward(saved, x)
        used.append(ws._buf.numel())
    q.qlin_poll_device_status()
    assert used == [blocks[0].workspace_bytes(M, training=True)] * 2
    assert used[0] == max(q.qlin_forward_gated_workspace(M, gated.w), q.qlin_forward_act_workspace(M, down.w),
                          q.qlin_backward_act_workspace(M, down.w), q.qlin_backward_gated_workspace(M, gated.w))


def test_reserve_under_a_capture_is_refused(q):  # noqa: F811
    """The graph's memory would be taken for the buffer of every later call."""
    from quantized_linear_layers_token_b200.ffn import Workspace
    ws = Workspace()
    ws.reserve(1 << 16)
    x = torch.zeros(8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x.add_(1)
        ws.reserve(1 << 10)  # large enough: nothing to do
        with pytest.raises(RuntimeError):
            ws.reserve(1 << 20)
    assert ws._buf.numel() == 1 << 16 and not ws._of_graphs
    g.replay()
    assert (x == 1).all()
