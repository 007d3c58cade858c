"""The feed-forward half of a transformer block on packed quantized weights:

    y = x + W_down (act(W_gate n(x)) * (W_up n(x)))

with n a layer norm or an RMS norm, for serving (one token and up) and for
fine-tuning over the frozen weights.  Four library calls forward
(:func:`qlin.qlin_norm_forward`, :func:`qlin.qlin_forward_gated`,
:func:`qlin.qlin_forward_act` with the residual), three backward; PyTorch
holds the memory and nothing else.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Callable

import torch

from . import qlin


@dataclass
class Saved:
    """What a training forward keeps for its backward pass."""
    x: torch.Tensor        # [M][D]
    mean: torch.Tensor     # [M], None for the RMS norm
    rstd: torch.Tensor     # [M]
    z: torch.Tensor        # [M][2 F] pre-activations, gate and up alternating
    s_gated: torch.Tensor  # the scales this forward quantized with
    s_down: torch.Tensor


class Workspace:
    """Device memory that the calls of one or of many blocks take turns on: one
    buffer, as large as the largest call so far needed.  Calls on it run one
    after the other on one stream, replays of captured calls among them.

    A buffer that a captured call uses is kept for this object's life, so a
    captured graph may be replayed as long as the object lives.  A capture
    cannot enlarge the buffer for the calls outside it: a call that finds it too
    small under a capture takes memory of its own in that graph.  So ``reserve``
    the largest size (``GatedFeedForward.workspace_bytes``), or run such a call
    once, before capturing.
    """

    def __init__(self, device: torch.device | str = "cuda"):
        self.device = device
        self._buf = None
        self._captured = []   # buffers that captured calls use
        self._of_graphs = []  # memory first made under a capture, one call's each

    def _new(self, nbytes: int) -> torch.Tensor:
        buf = torch.empty(max(nbytes, qlin.QLIN_WORKSPACE_HEAD), dtype=torch.uint8, device=self.device)
        buf[:qlin.QLIN_WORKSPACE_HEAD].zero_()
        return buf

    def reserve(self, nbytes: int) -> None:
        """Make the buffer at least this large (not under a capture)."""
        if self._buf is None or self._buf.numel() < nbytes:
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("a workspace cannot be enlarged under a capture: reserve it before")
            if self._buf is not None:
                self._buf.record_stream(torch.cuda.current_stream(self._buf.device))  # its last call may still run
            self._buf = self._new(nbytes)

    def get(self, nbytes: int) -> torch.Tensor:
        """A workspace of at least `nbytes` for the next call."""
        if not torch.cuda.is_current_stream_capturing():
            self.reserve(nbytes)
        elif self._buf is None or self._buf.numel() < nbytes:
            self._of_graphs.append(self._new(nbytes))  # its head zeroed by the graph, when it is replayed: for no other call
            return self._of_graphs[-1]
        elif not any(b is self._buf for b in self._captured):
            self._captured.append(self._buf)
        return self._buf

    def reset(self) -> None:
        """Ready again after a call gave up (QLIN_ERR_TIMEOUT): what has to be
        zero at the start of each buffer is zero-filled, in place."""
        for buf in [self._buf, *self._captured]:
            if buf is not None:
                buf[:qlin.QLIN_WORKSPACE_HEAD].zero_()


class GatedFeedForward:
    """`gated` is packed by ``PackedLayer.pack_gated`` ([D] -> 2 [F]), `down`
    by ``PackedLayer.pack`` ([F] -> [D]).  gamma, beta and the biases are fp32
    (`bias_gated` in the packed order); beta and the biases may be None.

    A training forward updates both momentum states (`s_gated`, `s_down`) and
    returns what its backward pass needs; several may be outstanding.  Calls run
    one after the other on one stream (they share a workspace), replays of
    captured calls among them.

    The blocks of a model take turns on one `workspace`, which they are given
    (by default each has its own: at 2048 tokens of LLaMA-2-70B's widths 1.2 GB).

    Data-parallel training: every rank's scales have to come from all ranks'
    tokens, or the replicas' states drift apart.  `reduce_max` combines a rank's
    fp32 vector of outlier column maxima with the other ranks' in place
    (``dp.max_over_ranks``); a training forward then calls it before each of its
    two quantizations, on every rank in the same order, a rank without tokens
    among them, and updates both states from the result, the same on every rank:
    the update over the unsharded batch.  Without it the states follow this
    process's tokens alone.

    After QLIN_ERR_TIMEOUT (``qlin.qlin_poll_device_status``) the outputs of the
    calls that gave up are undefined, and so is the `s_down` of a training
    forward among them: call ``reset`` and put back the states of before.
    """

    def __init__(self, gated: qlin.PackedLayer, down: qlin.PackedLayer, gamma, beta=None, bias_gated=None,
                 bias_down=None, kind: int = qlin.QLIN_NORM_RMS, eps: float = 1e-5, act: int = qlin.QLIN_ACT_SILU,
                 momentum: float = 0.9, workspace: Workspace | None = None,
                 reduce_max: Callable[[torch.Tensor], None] | None = None):
        if gated.K != down.N or gated.N != 2 * down.K:
            raise ValueError(f"gated [{gated.K}] -> [{gated.N}] and down [{down.K}] -> [{down.N}] do not fit together")
        self.gated, self.down = gated, down
        self.D, self.F = down.N, down.K
        self.gamma, self.beta, self.bias_gated, self.bias_down = gamma, beta, bias_gated, bias_down
        self.kind, self.eps, self.act, self.momentum = kind, eps, act, momentum
        dev = gated.buffer.device
        self.s_gated = torch.ones(gated.n_outlier, device=dev)
        self.s_down = torch.ones(down.n_outlier, device=dev)
        self.workspace = Workspace(dev) if workspace is None else workspace
        self.reduce_max = reduce_max

    def workspace_bytes(self, M: int, training: bool = False) -> int:
        """What the workspace holds for a forward of M tokens; with `training`,
        for its backward pass too."""
        n = max(qlin.qlin_forward_gated_workspace(M, self.gated.w), qlin.qlin_forward_act_workspace(M, self.down.w))
        return max(n, self._backward_bytes(M)) if training else n

    def _backward_bytes(self, M: int) -> int:
        return max(qlin.qlin_backward_act_workspace(M, self.down.w), qlin.qlin_backward_gated_workspace(M, self.gated.w),
                   qlin.qlin_norm_backward_workspace(M, self.D))

    def reset(self) -> None:
        """After a call gave up: the workspace is ready again (every block on it)."""
        self.workspace.reset()

    def _rows(self, t: torch.Tensor, name: str) -> int:
        if t.dim() != 2 or t.shape[1] != self.D:
            raise ValueError(f"{name} must be [M][{self.D}], got {tuple(t.shape)}")
        return t.shape[0]

    def _half(self, *shape):
        return torch.empty(shape, dtype=torch.float16, device=self.gated.buffer.device)

    def _update(self, x: torch.Tensor, M: int, layer: qlin.PackedLayer, s: torch.Tensor) -> bool:
        """Whether the layer's own call is to update its momentum state from
        its input x; with `reduce_max` it is done here, from all ranks' maxima."""
        if self.reduce_max is None:
            return True
        if layer.n_outlier > 0:
            cmax = torch.empty(layer.n_outlier, dtype=torch.float32, device=s.device)
            qlin.qlin_outlier_colmax(x, M, layer.w, cmax)
            self.reduce_max(cmax)
            qlin.qlin_momentum_update(layer.w, cmax, s, self.momentum)
        return False

    def forward(self, x: torch.Tensor, training: bool = False):
        """y [M][D] of x fp16 [M][D]; with `training`, (y, Saved)."""
        M = self._rows(x, "x")
        n, h, y = self._half(M, self.D), self._half(M, self.F), self._half(M, self.D)
        z = self._half(M, 2 * self.F) if training else None
        f32 = dict(dtype=torch.float32, device=n.device)
        mean = torch.empty(M, **f32) if training and self.kind == qlin.QLIN_NORM_LAYER else None
        rstd = torch.empty(M, **f32) if training else None
        qlin.qlin_norm_forward(x, M, self.D, self.kind, self.gamma, self.beta, self.eps, n, mean, rstd)
        ws = self.workspace.get(self.workspace_bytes(M))
        nws = ws.numel()
        update = training and self._update(n, M, self.gated, self.s_gated)
        qlin.qlin_forward_gated(n, M, self.gated.w, self.s_gated, self.momentum, update, h, ws, nws, act=self.act,
                                bias=self.bias_gated, Z=z)
        update = training and self._update(h, M, self.down, self.s_down)
        qlin.qlin_forward_act(h, M, self.down.w, self.s_down, self.momentum, update, y, ws, nws,
                              bias=self.bias_down, residual=x)
        if not training:
            return y
        return y, Saved(x, mean, rstd, z, self.s_gated.clone(), self.s_down.clone())

    def backward(self, saved: Saved, dy: torch.Tensor) -> dict:
        """Gradients of x and of the trainable vectors (None where there is
        no such vector): dx, dgamma, dbeta, dbias_gated, dbias_down."""
        M = self._rows(dy, "dy")
        if M != saved.x.shape[0]:
            raise ValueError(f"dy has {M} rows, the forward had {saved.x.shape[0]}")
        dev = self.gated.buffer.device
        dh, dn, dx = self._half(M, self.F), self._half(M, self.D), self._half(M, self.D)

        def like(v, n):
            return None if v is None else torch.empty(n, dtype=torch.float32, device=dev)

        dbg, dbd = like(self.bias_gated, 2 * self.F), like(self.bias_down, self.D)
        dgamma, dbeta = like(self.gamma, self.D), like(self.beta, self.D)
        ws = self.workspace.get(self._backward_bytes(M))
        nws = ws.numel()
        qlin.qlin_backward_act(self.down.w, dy, None, M, saved.s_down, dh, dbd, ws, nws)
        qlin.qlin_backward_gated(self.gated.w, dh, saved.z, M, saved.s_gated, dn, dbg, ws, nws, act=self.act)
        qlin.qlin_norm_backward(dn, saved.x, M, self.D, self.kind, self.gamma, saved.mean, saved.rstd, dy, dx, dgamma,
                                dbeta, ws, nws)
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta, "dbias_gated": dbg, "dbias_down": dbd}
