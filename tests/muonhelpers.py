"""Shared pieces of the tests of the orthogonalised update: the plain forms in
64 bits, and inputs.

Tolerance of a direction, in units of h = 2^-11, half a step of binary16: the
products of each step read X (twice for A = X X^T, once for B X), A (twice
for A A) and B, each rounded to binary16 once. To first order these enter the
step's result X' = a X + (b A + c A A) X with the weights |b| l (A and the two
X in it), 2 c l^2 (the same through A A) and |b l + c l^2| (B, and the X that
it multiplies), l = s^2, relative to |X'|. At the singular values where the
default steps end (s in 0.68 .. 1.14, X' about 1) the roundings add as
independent ones: sqrt(3 (|b| l)^2 + 3 (2 c l^2)^2 + 2 (b l + c l^2)^2) <=
sqrt(3 * 36 + 3 * 47 + 2 * 8) = 16 at the far end and 8.5 at l = 1/2, each
rounding's root mean square being h / 2 at most (its error is spread over
+-h of values between one and two steps): 8 h at worst, 4 h in the middle. A
step's error reaches the end through the later steps' slopes, |s' / s| <= 2
in that range with changing sign; steps whose results are below the range
weigh less by as much as l is smaller. 10 h = 4.9e-3 of the direction's
2-norm covers the sum. Outputs add their own half step.
"""
from __future__ import annotations

import torch

H = 2.0 ** -11
DIRECTION = 10 * H
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
QUINTIC = ((3.4445, -4.7750, 2.0315),) * 5


def direction64(u, coefficients=QUINTIC, eps=1e-7):
    """The polynomial in 64 bits on the last two axes, step by step."""
    x = u.double()
    turned = x.shape[-2] > x.shape[-1]
    if turned:
        x = x.mT
    norm = x.square().sum(dim=(-1, -2), keepdim=True).sqrt().clamp(min=eps)
    x = x / norm if eps > 0 else torch.where(norm > 0, x / norm, torch.zeros_like(x))
    for a, b, c in coefficients:
        g = x @ x.mT.contiguous()
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.mT if turned else x


def matrices(shape, kind="gauss", seed=0, scale=1.0):
    """FP32 test matrices (count, rows, cols) or (rows, cols)."""
    gen = torch.Generator().manual_seed(seed)
    g = torch.randn(shape, generator=gen)
    rows, cols = shape[-2:]
    r = max(1, min(rows, cols) // 8)
    if kind == "lowrank":     # exactly rank r, up to rounding
        left = torch.randn(*shape[:-1], r, generator=gen)
        right = torch.randn(*shape[:-2], r, cols, generator=gen)
        g = left @ right
    elif kind == "spiked":    # a few strong directions over noise a thousand times weaker
        left = torch.randn(*shape[:-1], 1, generator=gen)
        right = torch.randn(*shape[:-2], 1, cols, generator=gen)
        g = left @ right + 1e-3 * g
    elif kind == "outliers":
        g = torch.where(torch.rand(shape, generator=gen) < 0.01, 100 * g, g)
    return g * scale


def off(x, ref):
    """2-norm of the difference over that of ref, matrix by matrix: the worst."""
    d = (x.double().cpu() - ref.cpu()).flatten(-2).norm(dim=-1)
    n = ref.cpu().flatten(-2).norm(dim=-1)
    return float((d / n.clamp(min=1e-300)).max())


def lr_factor(kind, rows, cols):
    return {"none": 1.0, "original": max(1.0, rows / cols) ** 0.5,
            "match_rms_adamw": 0.2 * max(rows, cols) ** 0.5}[kind]
