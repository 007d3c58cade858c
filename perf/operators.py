"""The operators of the feed-forward half of a transformer block over frozen
quantized weights, as they are measured: a normalisation, the quantized
linear layer with bias, activation and residual in its epilogue, and the
gated block (both projections, the activation and the product in one GEMM),
each with its backward pass.

`own` selects the side: False computes every operator in elementary torch
operations in fp32, True calls the library's entry points."""
import math

import numpy as np
import torch

own = False

PC, G128, W8 = 0, 1, 2                                     # weight formats: INT4 per channel, INT4 g128, INT8
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")       # activation codes 0 .. 4
GAMMA = float(np.float32(0.9))                             # momentum of the outlier scales
EPS = float(np.float32(1e-5))


def _dev():
    return "cuda" if torch.cuda.is_available() else "cpu"


# ----------------------------------------------------------------- cases

def listed():
    return [
        # serving, one new token: the down projection adds its result to the residual stream
        dict(name="down 1 token residual", op="linear", M=1, K=11008, N=4096, nO=110, fmt=PC, act="none", bias=False,
             residual=True, train=False),
        # fine-tuning forward of a GELU MLP's first layer: bias, activation, the pre-activation kept, momentum updated
        dict(name="fc gelu train 1000", op="linear", M=1000, K=4096, N=11008, nO=205, fmt=W8, act="gelu_tanh",
             bias=True, residual=False, train=True),
        # a ragged batch of a small odd-sized layer with everything in the epilogue
        dict(name="odd relu residual 67", op="linear", M=67, K=1152, N=2064, nO=23, fmt=G128, act="relu", bias=True,
             residual=True, train=False),
        # its backward pass at a fine-tuning batch: input gradient and bias gradient
        dict(name="fc gelu backward 2048", op="linear_bwd", M=2048, K=4096, N=11008, nO=205, fmt=W8, act="gelu_tanh",
             dbias=True),
        # serving, 16 sequences: gate and up projections of a 70B block, one new token each
        dict(name="gated decode 16", op="gated", M=16, K=8192, F=28672, nO=82, fmt=G128, act="silu", bias=False,
             train=False),
        # a 7B block's prompt of 4096 tokens
        dict(name="gated prefill 4096", op="gated", M=4096, K=4096, F=11008, nO=41, fmt=PC, act="silu", bias=False,
             train=False),
        # a small odd gated block in fine-tuning: biases, pre-activations kept, momentum updated
        dict(name="gated odd train 45", op="gated", M=45, K=1184, F=1000, nO=59, fmt=W8, act="gelu", bias=True,
             train=True),
        # the 7B block's backward pass at a fine-tuning batch
        dict(name="gated backward 2048", op="gated_bwd", M=2048, K=4096, F=11008, nO=41, fmt=G128, act="silu",
             dbias=False),
        # a small odd gated block's backward pass with its bias gradient
        dict(name="gated backward odd 131", op="gated_bwd", M=131, K=1056, F=520, nO=0, fmt=PC, act="gelu_tanh",
             dbias=True),
        # serving, one new token: latency
        dict(name="rms norm 1 token", op="norm", M=1, K=4096, kind="rms", beta=False),
        # a long prompt in front of a 70B block
        dict(name="layer norm 8192", op="norm", M=8192, K=8192, kind="layer", beta=True),
        # fine-tuning: input, weight and bias gradients, joined with the residual branch's gradient
        dict(name="layer norm backward 4099", op="norm_bwd", M=4099, K=4096, kind="layer", beta=True, dres=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear_bwd", "gated", "gated_bwd", "norm", "norm_bwd"))
    M = max(1, _log_int(rng, 1, 8192))
    if op in ("norm", "norm_bwd"):
        c = dict(op=op, M=M, K=32 * _log_int(rng, 1, 512), kind=rng.choice(("layer", "rms")), beta=rng.random() < 0.5)
        if c["kind"] == "rms":
            c["beta"] = False
        while c["M"] * c["K"] > 8192 * 8192:
            c["M"] = max(1, c["M"] // 2)
        if op == "norm_bwd":
            c["dres"] = rng.random() < 0.5
        return c
    fmt = rng.choice((PC, G128, W8))
    K = 128 * _log_int(rng, 1, 86) if fmt == G128 else 32 * _log_int(rng, 2, 344)
    N = 16 * _log_int(rng, 2, 1376)
    while 2 * M * K * N > 7.0e11 or K * N > 1.2e8:
        M, N = max(1, M // 2), (N if M > 64 else max(32, N // 32 * 16))
    nO = int(round(rng.choice((0.0, 0.01, 0.02, 0.05)) * K))
    c = dict(op=op, M=M, K=K, nO=nO, fmt=fmt, act=rng.choice(ACTS if op.startswith("linear") else ACTS[1:]))
    if op.startswith("linear"):
        c["N"] = N
    else:
        c["F"] = max(8, N // 16 * 8)
    if op.endswith("_bwd"):
        c["dbias"] = rng.random() < 0.5
    else:
        c["bias"], c["train"] = rng.random() < 0.5, rng.random() < 0.5
        if op == "linear":
            c["residual"] = rng.random() < 0.5
    return c


# ----------------------------------------------------------------- inputs

def _weights(W, fmt):
    """The packed weights as values: the INT8 operand B [K][N] and the factor c' [N] with W ~ c' B."""
    if fmt == G128:
        K, N = W.shape
        g = (W.abs().reshape(K // 128, 128, N).amax(1).float() / 7).half().float()
        c = 7 * g.amax(0) / 127
        r = torch.where(c > 0, g / c, torch.zeros_like(g)).half().float()
        q = torch.where(g[:, None] > 0, W.reshape(K // 128, 128, N).float() / g[:, None], torch.zeros((), device=W.device))
        B = torch.round(torch.round(q).clamp_(-7, 7) * r[:, None])
        return B.reshape(K, N).to(torch.int8), c
    qmax = 127 if fmt == W8 else 7
    top = W.abs().amax(0).float()
    q = torch.round(W.float() * torch.where(top > 0, qmax / top, torch.zeros_like(top))).clamp_(-qmax, qmax)
    c = top / qmax
    return (q.to(torch.int8), c) if fmt == W8 else ((q * 16).to(torch.int8), c / 16)


def _inputs(case, seed):
    """Inputs of a case from its seed: activations with a few large outlier channels, weights N(0, 0.02^2),
    gradients N(0, 2^-14), as a model's layers see them."""
    dev = _dev()
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    n = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    op, M, K = case["op"], case["M"], case["K"]
    s = {"case": case}
    if op.startswith("norm"):
        spread = 1 + 30 * (torch.rand(K, generator=gen, device=dev) < 0.01).float()
        s["X"] = ((n(M, K) + 0.3) * spread).half()
        s["gamma"] = 1 + 0.1 * n(K)
        s["beta"] = 0.1 * n(K) if case["beta"] else None
        if op == "norm_bwd":
            x = s["X"].double()
            mean = x.mean(1) if case["kind"] == "layer" else torch.zeros(M, device=dev, dtype=torch.float64)
            s["mean"] = mean.float()
            s["rstd"] = (1 / torch.sqrt(((x - mean[:, None]) ** 2).mean(1) + EPS)).float()
            s["dY"] = (n(M, K) / 128).half()
            s["dres"] = (n(M, K) / 128).half() if case["dres"] else None
        return s
    gated = op.startswith("gated")
    N, nO, fmt = (2 * case["F"] if gated else case["N"]), case["nO"], case["fmt"]
    s["W"] = (n(K, N) * 0.02).half()
    s["O"] = torch.sort(torch.randperm(K, generator=gen, device=dev)[:nO]).values
    s["s"] = 1 + 7 * torch.rand(nO, generator=gen, device=dev)
    if op.endswith("_bwd"):
        s["Z"] = n(M, N).half()
        s["dY"] = (n(M, case["F"] if gated else N) / 128).half()
        return s
    X = n(M, K)
    X[:, s["O"]] *= 20 + 40 * torch.rand(nO, generator=gen, device=dev)
    s["X"] = X.half()
    s["bias"] = 0.2 * n(N) if case["bias"] else None
    s["residual"] = n(M, N).half() if case.get("residual") else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op, M, K, dev = case["op"], case["M"], case["K"], _dev()
    if op.startswith("norm"):
        if own:
            _own_norm(s)
        return s
    B, c = _weights(s["W"], case["fmt"])
    s["B"], s["c"] = B, c
    s["WO"] = s["W"][s["O"]].contiguous()
    s["wmax"] = s["WO"].abs().amax(1).float() if case["nO"] else torch.zeros(0, device=dev)
    if own:
        _own_weights(s)
    del s["W"]
    return s


def _own_norm(s):
    from quantized_linear_layers_token_b200 import qlin
    case = s["case"]
    M, K = s["X"].shape
    s["q"], s["kind"] = qlin, qlin.QLIN_NORM_LAYER if case["kind"] == "layer" else qlin.QLIN_NORM_RMS
    if case["op"] == "norm":
        s["Y"] = torch.empty_like(s["X"])
        s["mean"] = torch.empty(M, device="cuda") if case["kind"] == "layer" else None
        s["rstd"] = torch.empty(M, device="cuda")
        return
    s["mean"] = s["mean"] if case["kind"] == "layer" else None
    s["dX"], s["dgamma"] = torch.empty_like(s["X"]), torch.empty(K, device="cuda")
    s["dbeta"] = torch.empty(K, device="cuda") if case["beta"] else None
    s["nws"] = qlin.qlin_norm_backward_workspace(M, K)
    s["ws"] = qlin.empty_workspace(s["nws"])


def _same_codes(layer, B, fmt):
    """Lays the case's own weight codes out in the packed layer (the tiles of include/qlin.h): a weight that lies
    on the border between two codes may fall on either side of it in the packer."""
    if fmt == G128:  # quantized by divisions that round alike on both sides
        return
    (K, N), r = B.shape, torch.arange(128, device=B.device)[:, None]
    TN, KB = -(-N // 128), -(-K // 128)
    full = torch.zeros(TN * 128, KB * 128, dtype=torch.int8, device=B.device)
    full[:N, :K] = B.t()
    x = full.view(TN, 128, KB, 128).permute(0, 2, 1, 3)
    if fmt == PC:  # byte b of a word: input b in the low nibble, input 4 + b in the high one
        q = (x.reshape(TN, KB, 128, 16, 2, 4) >> 4) & 15
        x = (q[..., 0, :] | (q[..., 1, :] << 4)).reshape(TN, KB, 128, 64)
    n = x.shape[-1] // 16
    at = torch.arange(n, device=B.device) ^ ((r >> 1) & 3 if fmt == PC else r & 7)
    layer.view("codes").copy_(x.reshape(TN, KB, 128, n, 16)[:, :, r, at].reshape(-1).view(torch.uint8))


def _own_weights(s):
    from quantized_linear_layers_token_b200 import qlin
    case, M = s["case"], s["case"]["M"]
    gated, O = case["op"].startswith("gated"), s["O"].int().cpu().numpy()
    if gated:
        s["layer"] = qlin.PackedLayer.pack_gated(s["W"][:, 0::2].contiguous(), s["W"][:, 1::2].contiguous(), O, case["fmt"])
    else:
        s["layer"] = qlin.PackedLayer.pack(s["W"], O, case["fmt"])
    _same_codes(s["layer"], s["B"], case["fmt"])
    w, N = s["layer"].w, s["layer"].N
    s["q"], s["act"] = qlin, ACTS.index(case["act"])
    if case["op"].endswith("_bwd"):
        s["dX"] = torch.empty(M, case["K"], device="cuda", dtype=torch.float16)
        s["dbias"] = torch.empty(N, device="cuda") if case["dbias"] else None
        s["nws"] = (qlin.qlin_backward_gated_workspace if gated else qlin.qlin_backward_act_workspace)(M, w)
    else:
        s["Y"] = torch.empty(M, N // 2 if gated else N, device="cuda", dtype=torch.float16)
        s["Z"] = torch.empty(M, N, device="cuda", dtype=torch.float16) if case["train"] else None
        s["nws"] = (qlin.qlin_forward_gated_workspace if gated else qlin.qlin_forward_act_workspace)(M, w)
    s["ws"] = qlin.empty_workspace(s["nws"])
    del s["B"]  # the plain form's operand: the packed layer takes its place


# ----------------------------------------------------------------- plain forms

def _act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z * math.sqrt(0.5))
    if name == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        k = 2 * math.sqrt(2 / math.pi)
        p = 1 / (1 + torch.exp(-k * (z + 0.044715 * z * z * z)))
        return p + z * p * (1 - p) * k * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def _momentum(x, wmax, s):
    g = torch.full_like(s, GAMMA)
    beta = torch.where(wmax > 0, torch.clamp(torch.sqrt(x.abs().amax(0) / wmax), min=1), torch.ones_like(s))
    return g * s + (1 - g) * beta


def _preactivation(s, scales):
    x, O = s["X"].float(), s["O"]
    x[:, O] = x[:, O] / scales
    top = x.abs().amax(1, keepdim=True)
    q = torch.round(x * torch.where(top > 0, 127 / top, torch.zeros_like(top))).clamp(-127, 127)
    z = (q @ s["B"].float()) * s["c"] + (q[:, O] * (scales - 1)) @ s["WO"].float()
    z = z * (top / 127)
    return z if s["bias"] is None else z + s["bias"]


def _input_gradient(s, dz):
    O, scales = s["O"], s["s"]
    dx = (dz * s["c"]) @ s["B"].float().t()
    dx[:, O] = (dx[:, O] + (dz @ s["WO"].float().t()) * (scales - 1)) / scales
    return dx.half()


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op in ("linear", "gated"):
        scales = _momentum(s["X"][:, s["O"]].float(), s["wmax"], s["s"]) if case["train"] else s["s"]
        z = _preactivation(s, scales)
        if op == "linear":
            y = _act(case["act"], z)
            y = y if s["residual"] is None else y + s["residual"].float()
        else:
            y = _act(case["act"], z[:, 0::2]) * z[:, 1::2]
        return {"Y": y.half(), "Z": z.half(), "s": scales} if case["train"] else {"Y": y.half()}
    if op in ("linear_bwd", "gated_bwd"):
        z, dy = s["Z"].float(), s["dY"].float()
        if op == "linear_bwd":
            dz = dy * _act_grad(case["act"], z)
        else:
            g, u = z[:, 0::2], z[:, 1::2]
            dz = torch.stack([dy * u * _act_grad(case["act"], g), dy * _act(case["act"], g)], -1).reshape(z.shape)
        out = {"dX": _input_gradient(s, dz)}
        return {**out, "dbias": dz.sum(0)} if case["dbias"] else out
    x = s["X"].float()
    if op == "norm":
        mean = x.mean(1) if case["kind"] == "layer" else torch.zeros_like(x[:, 0])
        d = x - mean[:, None]
        rstd = 1 / torch.sqrt((d * d).mean(1) + EPS)
        y = d * rstd[:, None] * s["gamma"]
        y = (y if s["beta"] is None else y + s["beta"]).half()
        return {"Y": y, "mean": mean, "rstd": rstd} if case["kind"] == "layer" else {"Y": y, "rstd": rstd}
    dy = s["dY"].float()
    xhat = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["gamma"]
    inner = g - xhat * (g * xhat).mean(1, keepdim=True)
    if case["kind"] == "layer":
        inner = inner - g.mean(1, keepdim=True)
    dx = inner * s["rstd"][:, None]
    dx = (dx if s["dres"] is None else dx + s["dres"].float()).half()
    out = {"dX": dx, "dgamma": (dy * xhat).sum(0)}
    return {**out, "dbeta": dy.sum(0)} if case["beta"] else out


# ----------------------------------------------------------------- the library's calls

def _library(s):
    case, q = s["case"], s["q"]
    op, M, K = case["op"], case["M"], case["K"]
    if op == "linear":
        scales = s["s"].clone() if case["train"] else s["s"]
        q.qlin_forward_act(s["X"], M, s["layer"].w, scales, GAMMA, case["train"], s["Y"], s["ws"], s["nws"],
                           act=s["act"], bias=s["bias"], residual=s["residual"], Z=s["Z"])
        return {"Y": s["Y"], "Z": s["Z"], "s": scales} if case["train"] else {"Y": s["Y"]}
    if op == "gated":
        scales = s["s"].clone() if case["train"] else s["s"]
        q.qlin_forward_gated(s["X"], M, s["layer"].w, scales, GAMMA, case["train"], s["Y"], s["ws"], s["nws"],
                             act=s["act"], bias=s["bias"], Z=s["Z"])
        return {"Y": s["Y"], "Z": s["Z"], "s": scales} if case["train"] else {"Y": s["Y"]}
    if op in ("linear_bwd", "gated_bwd"):
        call = q.qlin_backward_act if op == "linear_bwd" else q.qlin_backward_gated
        call(s["layer"].w, s["dY"], s["Z"], M, s["s"], s["dX"], s["dbias"], s["ws"], s["nws"], act=s["act"])
        return {"dX": s["dX"], "dbias": s["dbias"]} if case["dbias"] else {"dX": s["dX"]}
    if op == "norm":
        q.qlin_norm_forward(s["X"], M, K, s["kind"], s["gamma"], s["beta"], EPS, s["Y"], s["mean"], s["rstd"])
        return {"Y": s["Y"], "mean": s["mean"], "rstd": s["rstd"]} if case["kind"] == "layer" else \
            {"Y": s["Y"], "rstd": s["rstd"]}
    q.qlin_norm_backward(s["dY"], s["X"], M, K, s["kind"], s["gamma"], s["mean"], s["rstd"], s["dres"], s["dX"],
                         s["dgamma"], s["dbeta"], s["ws"], s["nws"])
    out = {"dX": s["dX"], "dgamma": s["dgamma"]}
    return {**out, "dbeta": s["dbeta"]} if case["beta"] else out


def run(state):
    return _library(state) if own else _plain(state)


# ----------------------------------------------------------------- the definition in 64 bits

def _phi(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def _value_and_slope(name, z):
    """act(z) and act'(z) in fp64."""
    one = torch.ones_like(z)
    if name == "none":
        return z, one
    if name == "relu":
        return torch.clamp(z, min=0), torch.where(z > 0, one, 0 * one)
    if name == "gelu":
        return z * _phi(z), _phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2)
    sg = torch.sigmoid(z)
    return z * sg, sg + z * sg * (1 - sg)


def exact(case, seed):
    s = _inputs(case, seed)
    op, layer = case["op"], case.get("kind") == "layer"
    if op.startswith("norm"):
        x, gam = s["X"].double(), s["gamma"].double()
        if op == "norm":
            mu = x.sum(1, keepdim=True) / x.shape[1] if layer else torch.zeros_like(x[:, :1])
            r = ((x - mu).square().sum(1, keepdim=True) / x.shape[1] + EPS).rsqrt()
            y = (x - mu) * r * gam + (s["beta"].double() if s["beta"] is not None else 0)
            return {"Y": y, "mean": mu[:, 0], "rstd": r[:, 0]} if layer else {"Y": y, "rstd": r[:, 0]}
        dy, r = s["dY"].double(), s["rstd"].double()[:, None]
        h = (x - s["mean"].double()[:, None]) * r
        w = dy * gam
        K = x.shape[1]
        dx = r * (w - h * (w * h).sum(1, keepdim=True) / K - ((w.sum(1, keepdim=True) / K) if layer else 0))
        dx = dx + (s["dres"].double() if s["dres"] is not None else 0)
        out = {"dX": dx, "dgamma": torch.einsum("mk,mk->k", dy, h)}
        return {**out, "dbeta": dy.sum(0)} if case["beta"] else out
    B, c = _weights(s["W"], case["fmt"])
    O, sc = s["O"], s["s"].double()
    WO = s["W"][O].double()
    if op.endswith("_bwd"):
        z, dy = s["Z"].double(), s["dY"].double()
        if op == "linear_bwd":
            dz = dy * _value_and_slope(case["act"], z)[1]
        else:
            v, d = _value_and_slope(case["act"], z[:, 0::2])
            dz = torch.empty_like(z)
            dz[:, 0::2], dz[:, 1::2] = dy * z[:, 1::2] * d, dy * v
        # the effective weight: the outlier rows blended with their full-precision values
        We = B.double() * c.double()
        We[O] = (We[O] + (sc - 1)[:, None] * WO) / sc[:, None]
        out = {"dX": dz @ We.t()}
        return {**out, "dbias": dz.sum(0)} if case["dbias"] else out
    X32 = s["X"].float()
    s32 = s["s"]
    if case["train"]:
        peak, wm = X32[:, O].abs().amax(0).double(), s["W"][O].abs().amax(1).double() if len(O) else sc
        sc = GAMMA * sc + (1 - GAMMA) * torch.where(wm > 0, (peak / wm).sqrt().clamp(min=1), torch.ones_like(sc))
        # the codes below are whole numbers that the definition fixes through the fp32 state
        g32 = torch.tensor(GAMMA, dtype=torch.float32, device=s32.device)
        b32 = torch.where(wm > 0, (peak.float() / wm.float()).sqrt(), torch.ones_like(s32))
        s32 = g32 * s32 + (1 - g32) * torch.maximum(b32, torch.ones_like(s32))
    # the activation codes are whole numbers: the definition fixes them in fp32 (x / s, 127 / max, their product)
    X32[:, O] = X32[:, O] / s32
    top = X32.abs().amax(1)
    q = torch.round(X32 * torch.where(top > 0, 127 / top, torch.zeros_like(top))[:, None]).clamp(-127, 127).double()
    Z = q @ (B.double() * c.double()) + (q[:, O] * (s32.double() - 1)) @ WO
    Z = Z * (top.double() / 127)[:, None]
    if s["bias"] is not None:
        Z = Z + s["bias"].double()
    if op == "linear":
        Y = _value_and_slope(case["act"], Z)[0] + (s["residual"].double() if s["residual"] is not None else 0)
    else:
        Y = _value_and_slope(case["act"], Z[:, 0::2])[0] * Z[:, 1::2]
    return {"Y": Y, "Z": Z, "s": sc} if case["train"] else {"Y": Y}


# ----------------------------------------------------------------- work

def work(case):
    """What one pass cannot do without: each input read once, each output written once (fp16 activations, packed
    weights and scales, fp32 vectors), and the operations of the products."""
    op, M, K = case["op"], case["M"], case["K"]
    if op == "norm":
        return {"bytes": 4 * M * K + 4 * K * (2 if case["beta"] else 1) + 8 * M, "flops": 8 * M * K}
    if op == "norm_bwd":
        return {"bytes": (6 + 2 * case["dres"]) * M * K + 12 * K + 8 * M, "flops": 14 * M * K}
    gated = op.startswith("gated")
    N, nO = (2 * case["F"] if gated else case["N"]), case["nO"]
    weights = K * N // (1 if case["fmt"] == W8 else 2) + 4 * N + (K // 128 * N * 2 if case["fmt"] == G128 else 0)
    weights += nO * (2 * N + 12)
    if op.endswith("_bwd"):
        act = 2 * M * (case["F"] if gated else N) + 2 * M * N + 2 * M * K + (4 * N if case["dbias"] else 0)
        return {"bytes": weights + act, "flops": 2 * M * K * N}
    act = 2 * M * K + 2 * M * (case["F"] if gated else N) + (4 * N if case["bias"] else 0)
    act += 2 * M * N if case["train"] else 0
    act += 2 * M * N if case.get("residual") else 0
    return {"bytes": weights + act, "flops": 2 * M * K * N}
