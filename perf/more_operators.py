"""The loss of an output projection and the norms: the cases that are measured.

``loss`` is the softmax cross entropy of x W^T over a vocabulary, with the
gradients of x and W (``pass`` "gradients") or without ("loss"). ``norm`` is
layer norm or RMS norm over rows, forward, backward, or one after the other;
the residual form adds a residual to x first and its gradient to dx behind.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
IGNORE = -100


def listed():
    return [
        # the loss of one token, as a scorer asks for it: the weight is read once
        dict(name="loss 1 token", op="loss", **{"pass": "loss"}, tokens=1, hidden=2560,
             vocab=32000, dtype="bf16", ignored=0.0, reduction="sum", scale=1.0),
        # a handful of tokens of a small fine-tuning step: the weight's traffic decides
        dict(name="loss 24 tokens gradients", op="loss", **{"pass": "gradients"}, tokens=24,
             hidden=4096, vocab=128000, dtype="bf16", ignored=0.0, reduction="mean", scale=1.0),
        # odd sizes, loss-scaled half precision, prompts masked out
        dict(name="loss ragged fp16 masked", op="loss", **{"pass": "gradients"}, tokens=1003,
             hidden=2049, vocab=50021, dtype="fp16", ignored=0.4, reduction="mean", scale=1024.0),
        # evaluation over a validation batch
        dict(name="loss 4096 evaluated", op="loss", **{"pass": "loss"}, tokens=4096, hidden=2560,
             vocab=150000, dtype="bf16", ignored=0.1, reduction="mean", scale=1.0),
        # a training step at the 4B layer's width, a batch of padded sequences
        dict(name="loss 4096 x 2560 gradients", op="loss", **{"pass": "gradients"}, tokens=4096,
             hidden=2560, vocab=150000, dtype="bf16", ignored=0.1, reduction="mean", scale=1.0),
        # a training step at the 14B layer's width
        dict(name="loss 8192 x 5120 gradients", op="loss", **{"pass": "gradients"}, tokens=8192,
             hidden=5120, vocab=150000, dtype="bf16", ignored=0.0, reduction="mean", scale=1.0),
        # one sequence's last tokens through the final norm: nothing but latency
        dict(name="norm rms 4 tokens", op="norm", kind="rms", **{"pass": "forward"}, rows=4,
             heads=1, cols=2560, dtype="bf16", weight="bf16", bias=False, residual=False),
        # odd sizes, layer norm with a bias, half precision, FP32 weights
        dict(name="norm layer ragged fp16", op="norm", kind="layer", **{"pass": "both"}, rows=777,
             heads=1, cols=1027, dtype="fp16", weight="fp32", bias=True, residual=False),
        # the norm of each query head, inside the joint projection's rows
        dict(name="norm rms 40 heads of 128", op="norm", kind="rms", **{"pass": "both"}, rows=4096,
             heads=40, cols=128, dtype="bf16", weight="bf16", bias=False, residual=False),
        # a block's second norm at the 14B layer's width: residual, forward and backward
        dict(name="norm rms residual 8192x5120", op="norm", kind="rms", **{"pass": "both"},
             rows=8192, heads=1, cols=5120, dtype="bf16", weight="bf16", bias=False,
             residual=True),
        # layer norm's backward pass with both parameters' gradients, long batch
        dict(name="norm layer backward 32768", op="norm", kind="layer", **{"pass": "backward"},
             rows=32768, heads=1, cols=4096, dtype="bf16", weight="bf16", bias=True,
             residual=False),
        # FP32 activations
        dict(name="norm layer fp32 8192x2560", op="norm", kind="layer", **{"pass": "both"},
             rows=8192, heads=1, cols=2560, dtype="fp32", weight="fp32", bias=True,
             residual=False),
    ]


MOST_FLOPS = 6 * 8192 * 5120 * 150000
MOST_ELEMENTS = 32768 * 4096


def _spread(rng, low, high):
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    """Tokens 1 to 8192, widths 33 to 8192, vocabularies 300 to 160000; rows 1
    to 65536 of 16 to 32768 elements (of a few, a norm's gradient is what
    cancellation leaves); all over their logarithm, cut down to the largest
    listed cases."""
    if rng.random() < 0.5:
        tokens, hidden, vocab = _spread(rng, 1, 8192), _spread(rng, 33, 8192), \
            _spread(rng, 300, 160000)
        if rng.random() < 0.6:  # most models' widths are whole multiples
            hidden = max(64, hidden // 64 * 64)
        while 6 * tokens * hidden * vocab > MOST_FLOPS:
            tokens = max(1, tokens * 3 // 4)
        dtype, reduction = rng.choice(["bf16", "bf16", "fp16"]), rng.choice(["mean", "sum"])
        # half precision's gradients of a mean need a loss scale to stay in its range
        scale = 1024.0 if dtype == "fp16" and reduction == "mean" else rng.choice([1.0, 0.25])
        return dict(op="loss", **{"pass": rng.choice(["loss", "gradients", "gradients"])},
                    tokens=tokens, hidden=hidden, vocab=vocab, dtype=dtype,
                    ignored=rng.choice([0.0, 0.1, 0.5]), reduction=reduction, scale=scale)
    heads = rng.choice([1, 1, 1, rng.randint(2, 64)])
    cols = _spread(rng, 16, 32768 if heads == 1 else 512)
    rows = _spread(rng, 1, 65536 if heads == 1 else 8192)
    while rows * heads * cols > MOST_ELEMENTS:
        rows = max(1, rows * 3 // 4)
        cols = cols if rows > 1 else max(16, cols * 3 // 4)
    if rng.random() < 0.6 and cols > 64:
        cols = cols // 64 * 64
    kind = rng.choice(["rms", "layer"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    return dict(op="norm", kind=kind, **{"pass": rng.choice(["forward", "backward", "both"])},
                rows=rows, heads=heads, cols=cols, dtype=dtype,
                weight=rng.choice([dtype, "fp32"]),
                bias=kind == "layer" and rng.random() < 0.7,
                residual=heads == 1 and rng.random() < 0.4)


def _prepare_loss(case, gen):
    T, H, V, t = case["tokens"], case["hidden"], case["vocab"], TYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    weight = torch.empty(V, H, dtype=t, device="cuda")
    weight.normal_(0.0, 0.02, generator=gen)
    targets = torch.randint(0, V, (T,), device="cuda", generator=gen)
    # normalised hidden states that a trained head reads: their target's logit stands out by up
    # to 14, so that losses go from that of a guess to nearly none
    lift = torch.rand(T, 1, device="cuda", generator=gen) * (14.0 / (0.02 * H))
    x = randn(T, H) + lift * (weight[targets].float() / 0.02)
    x = (x / x.square().mean(dim=1, keepdim=True).sqrt()).to(t)
    targets[torch.rand(T, device="cuda", generator=gen) < case["ignored"]] = IGNORE
    return dict(x=x, weight=weight, targets=targets)


def _prepare_norm(case, gen):
    n, k, cols, t = case["rows"], case["heads"], case["cols"], TYPES[case["dtype"]]
    wt = TYPES[case["weight"]]

    def randn(*shape, spread=1.0):
        return torch.randn(*shape, device="cuda", generator=gen).mul_(spread)

    # the heads' rows lie inside a wider projection's: keys and values follow them
    shape, wide = ((n, cols), cols) if k == 1 else ((n, k, cols), (k + 16) * cols)

    def view(buffer):
        return buffer if k == 1 else buffer[:, :k * cols].unflatten(1, (k, cols))

    # token by token of different size, a few channels far larger than the others
    size = torch.exp(randn(n, 1, spread=0.5))
    outlier = torch.where(torch.rand(wide, device="cuda", generator=gen) < 0.01, 10.0, 1.0)
    s = dict(weight=(1.0 + randn(cols, spread=0.2)).to(wt),
             bias=randn(cols, spread=0.1).to(wt) if case["bias"] else None,
             x=view((randn(n, wide).mul_(size).mul_(outlier) + 0.05).to(t)),
             residual=randn(*shape).to(t) if case["residual"] else None)
    if case["pass"] != "forward":
        s["dy"] = randn(*shape, spread=1e-2).to(t)
        s["dsum"] = randn(*shape, spread=1e-2).to(t) if case["residual"] else None
    if case["pass"] == "backward":  # what the forward pass left
        if case["residual"]:
            s["x"] = (s["x"].float() + s["residual"].float()).to(t)
        s["stats"] = _statistics(s["x"].float(), case).reshape(_stats_shape(case))
    return s


def _stats_shape(case):
    return (2 if case["kind"] == "layer" else 1, case["rows"] * case["heads"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = _prepare_loss(case, gen) if case["op"] == "loss" else _prepare_norm(case, gen)
    state["case"] = case
    return state


def _eps(case):
    return 1e-5 if case["kind"] == "layer" else 1e-6


# ---- the plain forms ---------------------------------------------------------------------


def _plain_loss(state, gradients):
    case, y = state["case"], state["targets"]
    x, w = state["x"].float(), state["weight"].float()
    kept = y != IGNORE
    at = torch.where(kept, y, torch.zeros_like(y))[:, None]
    z = x @ w.T
    z = z - z.max(dim=1, keepdim=True).values
    e = torch.exp(z)
    total = e.sum(dim=1, keepdim=True)
    losses = torch.where(kept, torch.log(total[:, 0]) - z.gather(1, at)[:, 0], 0.0)
    count = kept.sum().clamp(min=1).double()
    loss = losses.double().sum()
    if case["reduction"] == "mean":
        loss = loss / count
    if not gradients:
        return {"loss": loss.float(), "losses": losses}
    g = e / total
    g.scatter_add_(1, at, torch.full_like(at, -1.0, dtype=torch.float32))
    c = case["scale"] * torch.where(kept, 1.0, 0.0)[:, None]
    if case["reduction"] == "mean":
        c = c / count.float()
    g = g * c
    return {"loss": loss.float(), "losses": losses, "dx": (g @ w).to(state["x"].dtype),
            "dweight": (g.T @ x).to(state["weight"].dtype)}


def _statistics(x, case):
    """(mean, rstd) of layer norm, (rstd) of RMS norm, in x's own number of bits."""
    mean = x.mean(dim=-1) if case["kind"] == "layer" else None
    d = x if mean is None else x - mean[..., None]
    rstd = 1.0 / torch.sqrt(d.square().mean(dim=-1) + _eps(case))
    return torch.stack([rstd] if mean is None else [mean, rstd])


def _normalised(x, stats):
    return (x if len(stats) == 1 else x - stats[0][..., None]) * stats[-1][..., None]


def _forward(x, w, b, case):
    stats = _statistics(x, case)
    y = _normalised(x, stats) * w
    return y if b is None else y + b, stats


def _backward(dy, x, w, stats, dsum, case):
    xh = _normalised(x, stats)
    g = dy * w
    dx = g - xh * (g * xh).mean(dim=-1, keepdim=True)
    if case["kind"] == "layer":
        dx = dx - g.mean(dim=-1, keepdim=True)
    dx = dx * stats[-1][..., None]
    axes = tuple(range(x.dim() - 1))
    # over the rows in 64 bits: these sums are as long as the batch
    return (dx if dsum is None else dx + dsum, (dy * xh).sum(dim=axes, dtype=torch.float64),
            dy.sum(dim=axes, dtype=torch.float64) if case["bias"] else None)


def _norm(state, bits):
    """The passes of a case in `bits` (a dtype), outputs not yet rounded."""
    def of(name):
        t = state.get(name)
        return None if t is None else t.to(bits)

    case, x, out = state["case"], of("x"), {}
    if case["pass"] != "backward":
        if case["residual"]:
            out["sum"] = x + of("residual")
            x = out["sum"].to(state["x"].dtype).to(bits)  # the norm of the sum as it is stored
        out["y"], stats = _forward(x, of("weight"), of("bias"), case)
        out["stats"] = stats.reshape(_stats_shape(case))
    else:
        stats = of("stats").reshape(-1, *x.shape[:-1])
    if case["pass"] != "forward":
        out["dx"], out["dweight"], out["dbias"] = _backward(
            of("dy"), x, of("weight"), stats, of("dsum"), case)
    return {k: v for k, v in out.items() if v is not None}


def _plain_norm(state):
    types = dict(stats=torch.float32, dweight=state["weight"].dtype, dbias=state["weight"].dtype)
    return {k: v.to(types.get(k, state["x"].dtype))
            for k, v in _norm(state, torch.float32).items()}


# ---- the framework's -----------------------------------------------------------------------


def _own_norm(state):
    import optimizer_step_layeradam_amd as la
    case, x, w, out = state["case"], state["x"], state["weight"], {}
    layer = case["kind"] == "layer"
    stats = state.get("stats")
    if case["pass"] != "backward":
        more = dict(eps=_eps(case), residual=state["residual"])
        if layer:
            got = la.layer_norm(x, w, state["bias"], **more)
        else:
            got = la.rms_norm(x, w, **more)
        if case["residual"]:
            out["sum"] = x = got[2]
        out["y"], out["stats"] = got[0], got[1]
        stats = got[1]
    if case["pass"] != "forward":
        if layer:
            out["dx"], out["dweight"], out["dbias"] = la.layer_norm_backward(
                state["dy"], x, w, stats, residual_grad=state["dsum"], bias_grad=case["bias"])
        else:
            out["dx"], out["dweight"] = la.rms_norm_backward(state["dy"], x, w, stats,
                                                             residual_grad=state["dsum"])
    return {k: v for k, v in out.items() if v is not None}


def _own_loss(state, gradients):
    import optimizer_step_layeradam_amd as la
    case = state["case"]
    losses = torch.empty(case["tokens"], dtype=torch.float32, device="cuda")
    more = dict(ignore_index=IGNORE, reduction=case["reduction"], losses=losses)
    if not gradients:
        loss = la.linear_cross_entropy(state["x"], state["weight"], state["targets"], **more)
        return {"loss": loss, "losses": losses}
    loss, dx, dweight = la.linear_cross_entropy_gradients(
        state["x"], state["weight"], state["targets"], grad_scale=case["scale"], **more)
    return {"loss": loss, "losses": losses, "dx": dx, "dweight": dweight}


def run(state):
    case = state["case"]
    if case["op"] == "loss":
        gradients = case["pass"] == "gradients"
        return _own_loss(state, gradients) if own else _plain_loss(state, gradients)
    return _own_norm(state) if own else _plain_norm(state)


def work(case):
    """Every input read once, every output written once; products of the
    tokens that count (the expected number of them)."""
    if case["op"] == "loss":
        T, H, V = case["tokens"], case["hidden"], case["vocab"]
        n = T * (1.0 - case["ignored"])
        each = 2 if case["pass"] == "gradients" else 1
        return {"bytes": round(each * 2 * (n * H + V * H) + 12 * T + 4),
                "flops": round((6 if each == 2 else 2) * n * H * V)}
    n, cols = case["rows"] * case["heads"], case["cols"]
    b, wb = (4 if case["dtype"] == "fp32" else 2), (4 if case["weight"] == "fp32" else 2)
    stats = 4 * n * (2 if case["kind"] == "layer" else 1)
    params = (2 if case["bias"] else 1) * wb * cols
    fwd = (2 + 2 * case["residual"]) * b * n * cols + params + stats
    bwd = (3 + case["residual"]) * b * n * cols + wb * cols + params + stats
    return {"bytes": {"forward": fwd, "backward": bwd, "both": fwd + bwd}[case["pass"]],
            "flops": n * cols * {"forward": 8, "backward": 14, "both": 22}[case["pass"]]}


# ---- in 64 bits ------------------------------------------------------------------------------


def _exact_loss(state):
    """Token by token from the definition, some hundred tokens at a time."""
    case, y = state["case"], state["targets"]
    w = state["weight"].double()
    V, H = w.shape
    gradients = case["pass"] == "gradients"
    count = max(1, int((y != IGNORE).sum()))
    c = case["scale"] / (count if case["reduction"] == "mean" else 1)
    losses = torch.zeros(case["tokens"], dtype=torch.float64, device="cuda")
    dx = torch.zeros(case["tokens"], H, dtype=torch.float64, device="cuda")
    dw = torch.zeros(V, H, dtype=torch.float64, device="cuda") if gradients else None
    for first in range(0, case["tokens"], 1024):
        rows = torch.nonzero(y[first:first + 1024] != IGNORE)[:, 0] + first
        if not len(rows):
            continue
        x, t = state["x"][rows].double(), y[rows]
        log_p = torch.mm(x, w.t())
        log_p -= torch.logsumexp(log_p, dim=1, keepdim=True)
        k = torch.arange(len(rows), device="cuda")
        losses[rows] = -log_p[k, t]
        if gradients:
            g = log_p.exp_()
            g[k, t] = torch.expm1(-losses[rows])
            dx[rows] = torch.mm(g, w) * c
            dw.addmm_(g.t(), x, alpha=c)
    loss = losses.sum() / (count if case["reduction"] == "mean" else 1)
    out = {"loss": loss, "losses": losses}
    return dict(out, dx=dx, dweight=dw) if gradients else out


def _exact_norm(state):
    """The forward pass as written; the backward pass as the derivative that
    differentiation of that forward pass gives."""
    case = state["case"]
    x = state["x"].double()
    w = state["weight"].double().requires_grad_()
    b = torch.zeros_like(w) if state["bias"] is None else state["bias"].double()
    b = b.detach().requires_grad_()
    out = {}
    if case["pass"] != "backward" and case["residual"]:
        out["sum"] = x + state["residual"].double()
        x = out["sum"].to(state["x"].dtype).double()
    x = x.contiguous().requires_grad_()
    centred = x - x.mean(dim=-1, keepdim=True) if case["kind"] == "layer" else x
    spread = torch.sqrt((centred ** 2).sum(dim=-1) / case["cols"] + _eps(case))
    y = centred / spread[..., None] * w + b
    if case["pass"] != "backward":
        out["y"] = y.detach()
        stats = [x.mean(dim=-1)] if case["kind"] == "layer" else []
        out["stats"] = torch.stack([s.detach() for s in stats + [1.0 / spread]]) \
            .reshape(_stats_shape(case))
    if case["pass"] != "forward":
        dx, dw, db = torch.autograd.grad(y, (x, w, b), state["dy"].double())
        out["dx"] = dx + state["dsum"].double() if case["residual"] else dx
        out["dweight"] = dw
        if case["bias"]:
            out["dbias"] = db
    return out


def exact(case, seed):
    state = prepare(case, seed)
    return _exact_loss(state) if case["op"] == "loss" else _exact_norm(state)
