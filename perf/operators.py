"""The orthogonalised update and the Muon step: the cases that are measured.

``orthogonalize`` replaces each matrix U by O = p(X): X_0 = U / max(||U||_F,
eps), five times X <- a X + (b A + c A A) X with A = X X^T (on the transpose
where the matrix is tall). ``muon_step`` is the optimizer step around it: the
sum of the gradient replicas, the unscale, the momentum, the orthogonalised
direction, the decayed step on the FP32 master and the 16-bit compute copy.

Matrices are written "COUNTxROWSxCOLS", several of them joined by commas: one
call takes them all, as an optimizer hands over a layer.
"""
import math

import torch

own = False

STEPS = 5
A, B, C = 3.4445, -4.7750, 2.0315
EPS = 1e-7
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# The matrices of the decoder layers in this repository's workloads.
LAYER_4B = "1x4096x2560,2x1024x2560,1x2560x4096,2x9728x2560,1x2560x9728"
LAYER_14B = "1x5120x5120,2x1024x5120,1x5120x5120,2x17408x5120,1x5120x17408"


def _matrices(case):
    return [tuple(int(x) for x in s.split("x")) for s in case["matrices"].split(",")]


def listed():
    return [
        # one head's square block alone: nothing but latency
        dict(name="orth one 64x64", op="orth", matrices="1x64x64", dtype="bf16", out="bf16"),
        # a query projection taken head by head: many wide, flat matrices
        dict(name="orth 40 heads 128x5120", op="orth", matrices="40x128x5120", dtype="bf16",
             out="bf16"),
        # odd sizes, FP32 directions (an optimizer's own momentum), wide and tall in one call
        dict(name="orth ragged fp32", op="orth", matrices="3x333x1001,2x1283x517,1x77x5",
             dtype="fp32", out="bf16"),
        # a mixture layer's stacked expert matrices
        dict(name="orth 64 experts 768x2048", op="orth", matrices="64x768x2048", dtype="bf16",
             out="bf16"),
        # the 4B layer's query projection, tall, in half precision
        dict(name="orth tall 4096x2560 fp16", op="orth", matrices="1x4096x2560", dtype="fp16",
             out="fp16"),
        # the 14B layer's down projection alone: one large matrix
        dict(name="orth 5120x17408", op="orth", matrices="1x5120x17408", dtype="bf16",
             out="bf16"),
        # the smallest layer, the first steps of a run: launches decide
        dict(name="muon tiny layer", op="muon", matrices="1x256x256,2x256x64,1x688x256", R=1,
             dtype="bf16", out="bf16", nesterov=True, unscale=1.0, scale="match_rms_adamw",
             lr=1e-5),
        # loss-scaled FP16 gradients, odd sizes, the flag on
        dict(name="muon ragged fp16", op="muon", matrices="1x1000x1500,2x129x2047,1x2049x511",
             R=2, dtype="fp16", out="fp16", nesterov=False, unscale=1.0 / 1024, scale="original",
             lr=2e-5),
        # stacked experts, one replica
        dict(name="muon 32 experts", op="muon", matrices="32x768x2048,32x2048x768", R=1,
             dtype="bf16", out="bf16", nesterov=True, unscale=1.0, scale="match_rms_adamw",
             lr=1e-4),
        # whole decoder layers with their replicas
        dict(name="muon 4B layer R=4", op="muon", matrices=LAYER_4B, R=4, dtype="bf16",
             out="bf16", nesterov=True, unscale=0.25, scale="match_rms_adamw", lr=1e-5),
        dict(name="muon 14B layer R=8", op="muon", matrices=LAYER_14B, R=8, dtype="bf16",
             out="bf16", nesterov=True, unscale=0.125, scale="match_rms_adamw", lr=1e-5),
    ]


def _flops(matrices):
    return sum(k * (15 * min(r, c) ** 2 * max(r, c) + 5 * min(r, c) ** 3) for k, r, c in matrices)


def draw(rng):
    """One to four groups of matrices, sides from 1 to 12000 (over their
    logarithm), stacks of up to 64, cut down to the cost of the 14B layer's
    share."""
    def side():
        return max(1, min(12000, round(math.exp(rng.uniform(0.0, math.log(12001.0))))))

    op = rng.choice(["orth", "muon"])
    groups = []
    # sizes are spread evenly, so the budget is spread too: small cases are drawn as often
    budget = math.exp(rng.uniform(math.log(2e9), math.log(5e12)))
    for _ in range(rng.randint(1, 4)):
        k, r, c = round(math.exp(rng.uniform(0.0, math.log(64.5)))), side(), side()
        while k > 1 and (_flops([(k, r, c)]) > budget or k * r * c > 6e7):
            k = (k + 1) // 2
        while _flops([(k, r, c)]) > budget or k * r * c > 6e7:
            r, c = max(1, r * 3 // 4), max(1, c * 3 // 4)
        groups.append((max(1, k), r, c))
    case = dict(op=op, matrices=",".join("%dx%dx%d" % g for g in groups))
    if op == "orth":
        case["dtype"] = rng.choice(["bf16", "fp16", "fp32"])
        case["out"] = rng.choice(["bf16", "fp16"])
    else:
        case.update(R=rng.randint(1, 8), dtype=rng.choice(["bf16", "fp16"]),
                    out=rng.choice(["bf16", "fp16"]), nesterov=rng.random() < 0.5,
                    unscale=rng.choice([1.0, 0.125, 1.0 / 1024]),
                    scale=rng.choice(["match_rms_adamw", "original", "none"]),
                    lr=rng.choice([1e-5, 2e-5, 1e-4]))
        if case["scale"] != "match_rms_adamw":
            # a direction of unscaled rows moves small matrices far: an ordinary rate for these
            case["lr"] = 1e-5
    return case


def _gradient(gen, shape, scale):
    """A gradient as layers have it: a few strong directions of falling
    weight, and noise below them."""
    k, rows, cols = shape
    rank = min(24, rows, cols)
    u = torch.randn(k, rows, rank, device="cuda", generator=gen)
    v = torch.randn(k, rank, cols, device="cuda", generator=gen)
    w = torch.arange(1, rank + 1, device="cuda", dtype=torch.float32) ** -0.7
    return torch.baddbmm(torch.randn(shape, device="cuda", generator=gen), u * w, v) \
        .mul_(scale)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    shapes, t = _matrices(case), TYPES[case["dtype"]]
    state = {"case": case}
    if case["op"] == "orth":
        state["x"] = [_gradient(gen, s, 1e-3).to(t) for s in shapes]
        state["out"] = [torch.empty(s, dtype=TYPES[case["out"]], device="cuda") for s in shapes]
        return state
    loss_scale = 1024.0 if case["unscale"] < 1e-2 else 1.0
    state["grads"], state["params"] = [], []
    for s in shapes:
        g = _gradient(gen, s, 1e-3 * loss_scale)
        state["grads"].append([
            (g + torch.randn(s, device="cuda", generator=gen).mul_(5e-4 * loss_scale)).to(t)
            for _ in range(case["R"])])
        del g
        state["params"].append((
            torch.randn(s, device="cuda", generator=gen).mul_(0.02),
            _gradient(gen, s, 2e-3),
            torch.empty(s, dtype=TYPES[case["out"]], device="cuda")))
    state["flag"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return state


def _hyper(case):
    return dict(lr=case["lr"], momentum=0.95, weight_decay=0.01, nesterov=case["nesterov"],
                grad_unscale=case["unscale"], lr_scale=case["scale"])


def _scale(kind, rows, cols):
    if kind == "match_rms_adamw":
        return 0.2 * math.sqrt(max(rows, cols))
    return math.sqrt(max(1.0, rows / cols)) if kind == "original" else 1.0


def _orthogonal(u):
    """The plain form of the direction: (k, rows, cols) in 32 bits."""
    norm = u.double().square().sum(dim=(1, 2), keepdim=True).sqrt()
    x = u / norm.clamp(min=EPS).float()
    tall = u.shape[1] > u.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    for _ in range(STEPS):
        g = torch.bmm(x, x.transpose(1, 2))
        x = A * x + torch.bmm(B * g + C * torch.bmm(g, g), x)
    return x.transpose(1, 2) if tall else x


def _plain_muon(state):
    case = state["case"]
    h = _hyper(case)
    for (p, m, w), grads in zip(state["params"], state["grads"]):
        g = grads[0].float()
        for r in grads[1:]:
            g = g + r.float()
        g = g * h["grad_unscale"]
        state["flag"].logical_or_(~torch.isfinite(g).all())
        m.mul_(h["momentum"]).add_(g)
        u = g + h["momentum"] * m if h["nesterov"] else m
        s = h["lr"] * _scale(h["lr_scale"], p.shape[1], p.shape[2])
        p.mul_(1.0 - h["lr"] * h["weight_decay"]).sub_(s * _orthogonal(u))
        w.copy_(p)


def run(state):
    case = state["case"]
    if case["op"] == "orth":
        if own:
            import optimizer_step_layeradam_amd as la
            la.orthogonalize(state["x"], state["out"])
        else:
            for x, o in zip(state["x"], state["out"]):
                o.copy_(_orthogonal(x.float()))
        return state["out"]
    if own:
        import optimizer_step_layeradam_amd as la
        if "layer" not in state:  # described once, as an optimizer keeps it
            state["layer"] = la.MuonLayer(state["params"], state["grads"])
        state["layer"].step(overflow_flag=state["flag"], **_hyper(case))
    else:
        _plain_muon(state)
    return {"params": state["params"], "flag": state["flag"]}


def work(case):
    """Symmetric products (X X^T and A A) counted as the half that has to be
    computed; every input read once, every output written once."""
    shapes = _matrices(case)
    n = sum(k * r * c for k, r, c in shapes)
    if case["op"] == "orth":
        per = (4 if case["dtype"] == "fp32" else 2) + 2
    else:
        per = 2 * case["R"] + 8 + 8 + 2
    return {"bytes": per * n, "flops": _flops(shapes)}


def _exact_direction(u):
    """The same polynomial in 64 bits, on the small Gram matrix: every factor
    is a polynomial in S = X_0 X_0^T, so S and the product Q of the factors
    are carried along, and O = Q X_0 at the end."""
    out = torch.empty_like(u)
    for i in range(u.shape[0]):
        x = u[i] if u.shape[1] <= u.shape[2] else u[i].T
        x = x / max(float(torch.linalg.matrix_norm(x)), EPS)
        s = x @ x.T
        q = None
        for _ in range(STEPS):
            f = torch.addmm(s, s, s, beta=B, alpha=C)
            f.diagonal().add_(A)
            q = f if q is None else f @ q
            s = f @ s @ f
        y = q @ x
        out[i] = y if u.shape[1] <= u.shape[2] else y.T
    return out


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "orth":
        return [_exact_direction(x.double()) for x in state["x"]]
    h = _hyper(case)
    params = []
    for (p, m, _), grads in zip(state["params"], state["grads"]):
        g = torch.zeros_like(p, dtype=torch.float64)
        for r in grads:
            g += r
        g *= h["grad_unscale"]
        m = m.double() * h["momentum"] + g
        o = _exact_direction(g + h["momentum"] * m if h["nesterov"] else m)
        s = h["lr"] * _scale(h["lr_scale"], p.shape[1], p.shape[2])
        p = p.double() * (1.0 - h["lr"] * h["weight_decay"]) - s * o
        params.append((p, m, p))
    return {"params": params, "flag": None}
