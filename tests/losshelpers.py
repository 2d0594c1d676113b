"""Shared pieces of the linear cross entropy's tests: inputs, the formulas in 64
bits, and bounds of the kernels' error counted from their roundings.

u = 2^-24 is half a step of binary32. Products of two 16-bit numbers are exact
in binary32; a matrix instruction adds 16 of them to its sum, each addition off
by at most a whole step (2 u), so a sum of K products is off by at most
2 u (K / 16 + 16) times the sum of their sizes. h is half a step of the tensors'
type.

- A logit is off by dz, its sum's error.
- lse: the largest dz, the exponentials (2 steps of the instruction, 2 u of the
  argument's rounding times its size, which e^-a a <= 0.37 keeps below 1) and
  their sums (at most 8 + 3 + 6 + 4 additions and the chunks that one thread adds,
  V / 64 / 256): below 64 u + V / 16384 u relative; rounding of the sum and of
  differences: 4 u (|largest logit| + |target's| + log V).
- g = exp(z - lse): relative error dz + dlse and those roundings again, 2^-11 for
  the binary16 exponential (with its own 2^-39 where it is below that format's
  range), h for its own rounding (2^-39 in binary16); the target's entry has its
  loss' error instead of the relative one.
- dx, dw: |error of g| times |w| or |x|, summed; the sum's error over K = V
  or tokens, with up to 64 parts added behind; three roundings of the factor; h.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def problem(tokens, hidden, vocab, dtype, seed=0, ignored=0.0, spread=1.0):
    """CPU x, weight, targets; logits of about `spread`, targets lifted."""
    gen = torch.Generator().manual_seed(seed)
    w = torch.randn(vocab, hidden, generator=gen)
    y = torch.randint(0, vocab, (tokens,), generator=gen)
    x = torch.randn(tokens, hidden, generator=gen) * (spread / hidden ** 0.5)
    x += w[y] * (torch.rand(tokens, 1, generator=gen) * 8.0 * spread / hidden)
    y[torch.rand(tokens, generator=gen) < ignored] = -100
    return x.to(dtype), w.to(dtype), y


class Truth:
    """The formulas in 64 bits (on the device of the inputs), with bounds."""

    def __init__(self, x, w, y, ignore=-100, mean=True, scale=1.0):
        dtype, (tokens, hidden), vocab = x.dtype, x.shape, w.shape[0]
        keep = y != ignore
        n = int(keep.sum())
        xk, yk, wd = x[keep].double(), y[keep].long(), w.double()
        z = torch.mm(xk, wd.t())
        top = z.max(1).values if n else z.sum(1)
        total = torch.exp(z - top[:, None]).sum(1)
        lse = top + total.log()
        rows = torch.arange(n, device=x.device)
        zt = z[rows, yk]
        self.losses = torch.zeros(tokens, dtype=torch.float64, device=x.device)
        self.losses[keep] = lse - zt
        div = max(n, 1) if mean else 1
        self.loss = self.losses.sum() / div
        c = abs(scale) / div
        g = torch.exp(z - lse[:, None])
        g[rows, yk] = torch.expm1(zt - lse)
        self.dx = torch.zeros(tokens, hidden, dtype=torch.float64, device=x.device)
        self.dx[keep] = scale / div * torch.mm(g, wd)
        self.dw = scale / div * torch.mm(g.t().contiguous(), xk)
        # bounds
        size = torch.mm(xk.abs(), wd.abs().t())
        dz = 2 * U * (hidden / 16 + 16) * (size.max(1).values if n else size.sum(1))
        biggest = z.abs().max(1).values if n else z.sum(1)
        off = 2 * dz + (64 + vocab / 16384) * U + 4 * U * (2 * biggest + torch.tensor(
            float(vocab)).log().item())
        self.off_losses = torch.zeros_like(self.losses)
        self.off_losses[keep] = off + U * (lse - zt).abs()
        self.off_loss = self.off_losses.sum() / div + 2 * U * self.loss.abs()
        half = HALF[dtype]
        dg = g.abs() * ((dz + off + 8 * U)[:, None] + 2.0 ** -11 + half * (1 + 2.0 ** -9)) \
            + 2.0 ** -38
        dg[rows, yk] += (off + U) * 1.01
        ga = g.abs()
        dx = c * (torch.mm(dg, wd.abs()) + U * (2 * (vocab / 16 + 16) + 64 + 8) *
                  torch.mm(ga, wd.abs()))
        self.off_dx = torch.zeros_like(self.dx)
        self.off_dx[keep] = dx
        self.off_dx += half * (self.dx.abs() + self.off_dx) + TINY[dtype]
        self.off_dx[~keep] = 0.0
        self.off_dw = c * (torch.mm(dg.t().contiguous(), xk.abs()) + U * (
            2 * (n / 16 + 16) + 8) * torch.mm(ga.t().contiguous(), xk.abs()))
        self.off_dw += half * (self.dw.abs() + self.off_dw) + TINY[dtype]
        if n == 0:
            self.off_dw.zero_()

    def check(self, loss=None, losses=None, dx=None, dw=None):
        for got, want, off, what in ((loss, self.loss, self.off_loss, "loss"),
                                     (losses, self.losses, self.off_losses, "losses"),
                                     (dx, self.dx, self.off_dx, "dx"),
                                     (dw, self.dw, self.off_dw, "dweight")):
            if got is None:
                continue
            d = (got.double().to(want.device) - want).abs()
            bad = ~(d <= off)
            assert not bool(bad.any()), (what, int(bad.sum()), bad.numel(),
                                         float((d / off.clamp(min=1e-300)).max()))
