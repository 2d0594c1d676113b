"""How far directions are from the polynomial in 64 bits, in 32 bits and on the
spectra that are hardest on them: one singular value far above the others, so
that what the others contribute to S = X X^T lies in its last bits.

The direction comes out in FP32 as the step of a master of zeros: with lr 1, no
scale, no decay and a momentum buffer of twice the matrix at momentum 1/2, whose
product is exact.

Tolerance of the narrow form (short side m in 17 .. 128), which iterates S in
numbers of 22 bits: an error E in S enters a step's factor a + b S + c S^2 as b E, beside a,
and grows by a^2 per step while S is small, so that the result is off by |b| / a
(1 + a^2 + a^4 + a^6 + a^8) = 3.0e4 times its part along each small singular
direction. Several roundings of half a step of 22 bits at most, adding as
independent ones, make E's norm about one step, 2^-22 of S's; spread over m
directions that is 2^-22 3.0e4 / m^(1/2) = 7.2e-3 / m^(1/2) of the result's norm.

Short sides up to 16 are iterated in 64 bits, with coefficients of 32: each is off
by half a step, 2^-24 of it, at most, and a step's result by 2^-24 (a s + |b| s^3 + c
s^5) more than the slope makes of the step before. The largest sum of these over
all singular values, beside the result's, is the bar, and a rounding to FP32.

The step-by-step form rounds X as the products read it, A and B off their
diagonals to binary16, with a root mean square of 2^-11 / 3^(1/2) of a value at the
low end of its binade and 0.735 times that over a binade. For a singular value s of
X and l = s^2, to first order, an X off by a part d moves the step's result by s (b
l + c l^2 + 2 (b l + 2 c l^2)) d, the last step's by a s d more (it reads X in 16
bits in its linear term too), an A by s (b l + 2 c l^2) d, a B by s (b l + c l^2) d.
These add as independent ones to what the slope makes of the step before. The
root mean square over the matrix's singular values is the bar: the roundings of
many elements move each of them by less than those of one number would.
"""
import pytest
import torch

import optimizer_step_layeradam_amd as la
from muonhelpers import direction64, matrices

pytestmark = pytest.mark.gpu

A, B, _ = la.NEWTON_SCHULZ[0]
GROWTH = abs(B) / A * sum(A ** (2 * k) for k in range(5))


def narrow_bar(m):
    return 2.0 ** -22 * GROWTH / m ** 0.5


def tiny_bar():
    a, b, c = la.NEWTON_SCHULZ[0]
    s = torch.logspace(-9, 0, 200001, dtype=torch.float64)
    e = torch.zeros_like(s)
    for _ in range(5):
        e = (a + 3 * b * s ** 2 + 5 * c * s ** 4).abs() * e + \
            2.0 ** -24 * (a * s - b * s ** 3 + c * s ** 5)
        s = (a * s + b * s ** 3 + c * s ** 5).abs()
    return float((e / s).max()) + 2.0 ** -24


def wide_bar(u):
    """Of the worst matrix in the stack u."""
    a, b, c = la.NEWTON_SCHULZ[0]
    s = torch.linalg.svdvals(u.double().cpu())
    s = s / s.norm(dim=-1, keepdim=True)
    v = torch.zeros_like(s)
    unit = 0.735 * 2.0 ** -11 / 3 ** 0.5
    for k in range(5):
        p, q = b * s ** 2 + c * s ** 4, b * s ** 2 + 2 * c * s ** 4
        of_x = p + 2 * q + (a if k == 4 else 0.0)
        v = (a + p + 2 * q) ** 2 * v + (unit * s) ** 2 * (of_x ** 2 + q ** 2 + p ** 2)
        s = (a * s + p * s).abs()
    return float((v.sum(dim=-1) / s.square().sum(dim=-1)).sqrt().max())


def dominated(shape, kind, eps, seed):
    """(count, rows, cols): a matrix of rank one and noise eps times as strong."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*s):
        return torch.randn(s, device="cuda", generator=gen)

    k, r, c = shape
    noise = randn(k, r, c)
    if kind == "constant":
        return 1 + eps * noise
    if kind == "rank one":
        return randn(k, r, 1) * randn(k, 1, c) + eps * noise
    if kind == "column":  # of the long side: S_0's first 64 terms outweigh the rest
        strong = (max(r, c) ** 0.5) / eps
        if r <= c:
            noise[:, :, 0] += strong
        else:
            noise[:, 0, :] += strong
        return noise
    return noise


def direction(u, *beside):
    params = [(torch.zeros_like(x), (2 * x).contiguous()) for x in (u, *beside)]
    grads = [[torch.zeros_like(x, dtype=torch.bfloat16)] for x in (u, *beside)]
    la.muon_step(params, grads, lr=1.0, momentum=0.5, nesterov=False, lr_scale="none")
    return -params[0][0]


def worst(u, *beside):
    want = direction64(u)
    d = (direction(u, *beside).double() - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)
    return float(d.max())


KINDS = [("constant", 0.03), ("constant", 0.01), ("constant", 0.001), ("rank one", 0.01),
         ("column", 0.01), ("noise", 1.0)]

# Long sums by one workgroup a matrix and in parts, wide and tall, sides of 64 and 128.
NARROW = [(520, 17, 2000), (520, 64, 5120), (513, 4000, 33), (1, 20, 100000), (3, 64, 12000),
          (8, 100, 3000), (2, 128, 30000), (1, 9000, 65), (40, 64, 64), (40, 17, 17)]


@pytest.mark.parametrize("kind,eps", KINDS)
@pytest.mark.parametrize("shape", NARROW, ids=str)
def test_narrow(shape, kind, eps):
    got, bar = worst(dominated(shape, kind, eps, sum(shape))), narrow_bar(min(shape[1:]))
    print(f"  off {got:.2e} (bar {bar:.2e})", flush=True)
    assert got <= bar


# Whole and in parts, squares, vectors, tall and wide, the largest side.
TINY = [(600, 2, 2), (300, 3, 5), (40, 16, 16), (7, 1, 1), (1, 1, 40000), (3, 2, 12000),
        (520, 4, 20000), (5, 30000, 7), (1, 3, 1048576), (2, 513, 16), (2, 16, 512), (9, 9, 200),
        (2, 13, 4)]


@pytest.mark.parametrize("kind,eps", KINDS)
@pytest.mark.parametrize("shape", TINY, ids=str)
def test_tiny(shape, kind, eps):
    got, bar = worst(dominated(shape, kind, eps, sum(shape))), tiny_bar()
    print(f"  off {got:.2e} (bar {bar:.2e})", flush=True)
    assert got <= bar


@pytest.mark.parametrize("shape", [(2, 2), (3, 2, 300), (16, 30), (150, 9)], ids=str)
def test_tiny_beside_wide(shape):
    """A large matrix in the same call does not change how a tiny one is done."""
    u = dominated((1, *shape)[-3:], "rank one", 0.01, 3).view(shape)
    big = dominated((1, 200, 300), "noise", 1.0, 4)[0]
    alone = la.orthogonalize(u)
    for together in (la.orthogonalize([u, big])[0], la.orthogonalize([big, u])[1]):
        assert torch.equal(alone.view(torch.int16), together.view(torch.int16))


SPECTRA = ["gauss", "lowrank", "spiked", "outliers"]


@pytest.mark.parametrize("kind", SPECTRA)
@pytest.mark.parametrize("shape", [(255, 257), (129, 1500), (300, 129), (513, 515), (3, 130, 200),
                                   (2, 700, 300)], ids=str)
def test_wide_spectra(shape, kind):
    u = matrices(shape, kind, seed=sum(shape)).cuda()
    u = u if u.dim() == 3 else u[None]
    got, bar = worst(u), wide_bar(u)
    print(f"  off {got:.2e} (bar {bar:.2e})", flush=True)
    assert got <= bar


@pytest.mark.parametrize("kind", SPECTRA)
@pytest.mark.parametrize("shape", [(31, 33), (65, 63), (64, 64), (100, 260), (128, 128),
                                   (7, 33, 70), (5, 17, 1030), (3, 1000, 24)], ids=str)
def test_narrow_spectra_alone_and_beside_a_wide_matrix(shape, kind):
    u = matrices(shape, kind, seed=sum(shape)).cuda()
    u = u if u.dim() == 3 else u[None]
    got, bar = worst(u), narrow_bar(min(u.shape[1:]))
    print(f"  off {got:.2e} (bar {bar:.2e})", flush=True)
    assert got <= bar
    wide = matrices((1, 200, 300), seed=1).cuda()  # in whose launches small stacks share
    got, bar = worst(u, wide), max(bar, wide_bar(u))
    print(f"  off {got:.2e} (bar {bar:.2e})", flush=True)
    assert got <= bar
