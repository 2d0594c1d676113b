"""Shared pieces of the norms' tests: inputs, the formulas in 64 bits, and
bounds of the kernels' error counted from their roundings.

u = 2^-24 is half a step of binary32. A sum over a row is a tree whose longest
chain has depth(cols) additions: a lane adds the elements it holds, lanes and
waves add each other's. Each addition rounds its partial sum, so the sum is off
by at most depth u times the sum of the absolute values. Terms are counted to
first order; the second is below them by u itself.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# half of the smallest spacing, where a rounding is no longer relative
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def depth(cols):
    """Additions one after the other in a row's sum: up to 32 elements a lane in
    registers, cols / 1024 of them where rows are long, then 6 exchanges and up
    to 16 waves."""
    return max(32, -(-cols // 1024) + 8) + 6 + 16


def inputs(rows, cols, dtype, seed=0, offset=0.5):
    """A CPU tensor whose rows differ in size, with a few large channels."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=gen)
    x *= torch.exp(torch.randn(rows, 1, generator=gen))
    x *= torch.where(torch.rand(cols, generator=gen) < 0.05, 20.0, 1.0)
    return (x + offset).to(dtype)


def params(cols, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed + 1000)
    return (1 + 0.3 * torch.randn(cols, generator=gen)).to(dtype), \
        (0.5 * torch.randn(cols, generator=gen)).to(dtype)


def forward64(s, w, b, eps, layer):
    """y, mean, rstd of rows s in 64 bits."""
    s = s.double()
    mean = s.mean(-1) if layer else torch.zeros_like(s[..., 0])
    rstd = 1.0 / ((s - mean[..., None]).square().mean(-1) + eps).sqrt()
    y = (s - mean[..., None]) * rstd[..., None]
    if w is not None:
        y = y * w.double()
    return (y if b is None else y + b.double()), mean, rstd


def forward_bound(s, w, b, eps, layer, y, mean, rstd, dtype):
    """|error| of y, mean and rstd at most, element by element."""
    s = s.double()
    d = depth(s.shape[-1])
    w = torch.ones_like(s[..., :1]) if w is None else w.double().abs()
    b = 0.0 if b is None else b.double().abs()
    size = s.abs().mean(-1)
    off_mean = (d + 2) * U * size if layer else torch.zeros_like(size)
    # the squares: 2 roundings each and the difference's, the sum's, the mean's,
    # eps', the root's and the quotient's; the mean's own error enters squared
    off_rstd = rstd * ((d + 6) / 2 + 3) * U + rstd ** 3 * off_mean ** 2
    h = (s - mean[..., None]).abs() * rstd[..., None]
    off_y = w * rstd[..., None] * off_mean[..., None] + h * w * (
        (off_rstd / rstd)[..., None] + 4 * U) + 2 * U * (h * w + b)
    return off_y + HALF[dtype] * (y.abs() + off_y) + TINY[dtype], \
        off_mean + U * mean.abs(), off_rstd + U * rstd


def backward64(dy, s, w, mean, rstd, layer, dsum=None):
    """dx, dweight, dbias in 64 bits, from the statistics as given."""
    dy, s = dy.double(), s.double()
    h = (s - mean.double()[..., None]) * rstd.double()[..., None]
    g = dy if w is None else dy * w.double()
    dx = g - h * (g * h).mean(-1, keepdim=True)
    if layer:
        dx = dx - g.mean(-1, keepdim=True)
    dx = dx * rstd.double()[..., None]
    cols = dy.shape[-1]
    return dx if dsum is None else dx + dsum.double(), (dy * h).reshape(-1, cols).sum(0), \
        dy.reshape(-1, cols).sum(0)


def backward_bound(dy, s, w, mean, rstd, layer, dx, dw, db, dsum, dtype, grad_dtype):
    """|error| of dx, dweight and dbias at most."""
    dy, s, mean, rstd = dy.double(), s.double(), mean.double(), rstd.double()
    cols, rows = s.shape[-1], dy[..., 0].numel()
    d = depth(cols)
    r = rstd[..., None]
    h = (s - mean[..., None]).abs() * r
    # the difference and the product: two roundings
    off_h = 2 * U * h + U * h
    g = (dy if w is None else dy * w.double()).abs()
    mg = g.mean(-1, keepdim=True) if layer else 0.0
    mgh = (g * h).mean(-1, keepdim=True)
    off_mg = (d + 3) * U * mg
    off_mgh = (d + 4) * U * mgh + (g * off_h).mean(-1, keepdim=True)
    inner = g + mg + h * mgh
    off = r * (off_mg + h * off_mgh + off_h * mgh + 5 * U * inner)
    if dsum is not None:
        off = off + U * (r * inner + dsum.double().abs())
    # a part's rows one after the other (or in up to 64 groups), then the parts in 32
    # chains: at most rows / 512 + 64 rows in a part, 64 groups, 16 parts a chain, 32 chains
    chain = -(-rows // 512) + 64 + 64 + 16 + 32

    def over_rows(t):
        return t.reshape(-1, cols).sum(0)

    off_dw = (chain + 1) * U * over_rows(dy.abs() * h) + over_rows(dy.abs() * off_h)
    off_db = chain * U * over_rows(dy.abs())
    return off + HALF[dtype] * (dx.abs() + off) + TINY[dtype], \
        off_dw + HALF[grad_dtype] * (dw.abs() + off_dw) + TINY[grad_dtype], \
        off_db + HALF[grad_dtype] * (db.abs() + off_db) + TINY[grad_dtype]


def within(got, want, bound, what):
    off = (got.double().cpu() - want.cpu()).abs()
    bad = ~(off <= bound.cpu())
    assert not bad.any(), (what, int(bad.sum()), float((off / bound.cpu()).max()))
