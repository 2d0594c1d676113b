"""The linear cross entropy on the GPU against its formulas in 64 bits, to
bounds counted from their roundings (tests/losshelpers.py): sizes that are no
whole tile, types, masks, pieces, strides, and what a call may not do."""
import pytest
import torch

import optimizer_step_layeradam_amd as la
from losshelpers import Truth, problem
from normhelpers import U

pytestmark = pytest.mark.gpu
BF, H = torch.bfloat16, torch.float16
NAN = float("nan")


def run(x, w, y, mean=True, scale=1.0, **kw):
    with torch.cuda.stream(kw.get("stream")):  # None: the current one
        losses = torch.full((y.numel(),), 9.0, device="cuda")
    loss, dx, dw = la.linear_cross_entropy_gradients(
        x, w, y, reduction="mean" if mean else "sum", grad_scale=scale, losses=losses, **kw)
    return loss, losses, dx, dw


def workspace(tokens, hidden, vocab, columns, packed=False):
    need = la.linear_cross_entropy_workspace_bytes(tokens, hidden, vocab, piece_columns=columns,
                                                   packed=packed)
    return torch.empty(need, dtype=torch.uint8, device="cuda")


SIZES = [(1, 64, 300), (1, 1, 1), (3, 64, 1), (5, 33, 77), (64, 64, 256), (65, 100, 1000),
         (130, 129, 515), (200, 320, 1030), (257, 128, 5000), (33, 2049, 700), (300, 192, 9001),
         (24, 512, 20000)]


@pytest.mark.parametrize("ignored", [0.0, 0.4])
@pytest.mark.parametrize("dtype", [BF, H])
@pytest.mark.parametrize("tokens,hidden,vocab", SIZES)
def test_against_formulas(tokens, hidden, vocab, dtype, ignored):
    x, w, y = problem(tokens, hidden, vocab, dtype, 1, ignored)
    x, w, y = x.cuda(), w.cuda(), y.cuda()
    scale = 64.0 if dtype == H else 1.0
    truth = Truth(x, w, y, mean=True, scale=scale)
    truth.check(*run(x, w, y, True, scale))
    losses = torch.empty(tokens, device="cuda")
    loss = la.linear_cross_entropy(x, w, y, losses=losses)
    truth.check(loss, losses)


@pytest.mark.parametrize("dtype", [BF, H])
@pytest.mark.parametrize("columns", [256, 512, 2048])
def test_pieces(columns, dtype):
    tokens, hidden, vocab = 150, 192, 3001
    x, w, y = (t.cuda() for t in problem(tokens, hidden, vocab, dtype, 2, 0.2))
    truth = Truth(x, w, y, mean=False, scale=0.5)
    truth.check(*run(x, w, y, False, 0.5, workspace=workspace(tokens, hidden, vocab, columns)))


def test_large_logits():
    """Logits of some hundreds: no exponential overflows, none is lost early."""
    for dtype in (BF, H):
        x, w, y = (t.cuda() for t in problem(100, 256, 2000, dtype, 3, 0.0, 40.0))
        Truth(x, w, y, mean=False).check(*run(x, w, y, False))


def test_well_predicted_tokens():
    """1 - p of a target with p near 1 keeps its bits: dx and the losses are small
    and still right, which the bound relative to the entry asks for."""
    x, w, y = (t.cuda() for t in problem(64, 512, 1500, BF, 4))
    x = (w[y].float() * (18.0 / 512)).to(BF)
    truth = Truth(x, w, y, mean=False)
    assert float(truth.losses.max()) < 1e-3
    truth.check(*run(x, w, y, False))


def test_more_axes_strides_and_index_types():
    tokens, hidden, vocab = 60, 128, 700
    x, w, y = (t.cuda() for t in problem(tokens, hidden, vocab, BF, 5, 0.2))
    truth = Truth(x, w, y)
    # rows inside wider ones, at an odd element
    wide = torch.full((tokens, hidden + 9), 5.0, dtype=BF, device="cuda")
    wide[:, 3:3 + hidden] = x
    wide_w = torch.full((vocab, hidden + 7), 5.0, dtype=BF, device="cuda")
    wide_w[:, 1:1 + hidden] = w
    dx = torch.full_like(wide, 5.0)
    dw = torch.full_like(wide_w, 5.0)
    got = run(wide[:, 3:3 + hidden], wide_w[:, 1:1 + hidden], y, dx=dx[:, 3:3 + hidden],
              dweight=dw[:, 1:1 + hidden])
    truth.check(*got)
    assert bool((dx[:, :3] == 5).all()) and bool((dx[:, 3 + hidden:] == 5).all())
    assert bool((dw[:, :1] == 5).all()) and bool((dw[:, 1 + hidden:] == 5).all())
    # rows inside wider ones, aligned: read as they lie
    wide_w = torch.full((vocab, hidden + 64), NAN, dtype=BF, device="cuda")
    wide_w[:, :hidden] = w
    truth.check(*run(x, wide_w[:, :hidden], y.int()))
    # batch by sequence
    loss, losses, dx, dw = run(x.reshape(4, 15, hidden), w, y.reshape(4, 15))
    assert dx.shape == (4, 15, hidden)
    truth.check(loss, losses, dx.reshape(tokens, hidden), dw)
    # one row for all tokens
    one = x[:1].expand(tokens, hidden)
    Truth(one, w, y).check(*run(one, w, y))


@pytest.mark.parametrize("columns", [0, 256])
def test_nothing_counts(columns):
    x, w, y = (t.cuda() for t in problem(70, 64, 600, BF, 6, 1.1))
    more = dict(workspace=workspace(70, 64, 600, columns)) if columns else {}
    dx, dw = torch.full_like(x, 3), torch.full_like(w, 3)
    loss, losses, _, _ = run(x, w, y, dx=dx, dweight=dw, **more)
    assert float(loss) == 0.0
    for t in (losses, dx, dw):
        assert bool((t == 0).all())


def test_no_tokens():
    w = torch.randn(500, 64, device="cuda").to(BF)
    x, y = torch.empty(0, 64, dtype=BF, device="cuda"), torch.empty(0, dtype=torch.int64,
                                                                    device="cuda")
    loss, dx, dw = la.linear_cross_entropy_gradients(x, w, y)
    assert float(loss) == 0.0 and dx.shape == (0, 64) and bool((dw == 0).all())
    assert float(la.linear_cross_entropy(x, w, y, reduction="sum")) == 0.0


@pytest.mark.parametrize("bad", [NAN, float("inf")])
@pytest.mark.parametrize("columns", [0, 256])
def test_ignored_rows_reach_nothing(columns, bad):
    tokens, hidden, vocab = 140, 128, 900
    x, w, y = (t.cuda() for t in problem(tokens, hidden, vocab, BF, 7, 0.5))
    more = dict(workspace=workspace(tokens, hidden, vocab, columns)) if columns else {}
    want = run(x, w, y, **more)
    x[y == -100] = bad
    for p, q in zip(run(x, w, y, **more), want):
        assert torch.equal(p, q)


def test_ignore_index_may_be_a_word():
    x, w, y = (t.cuda() for t in problem(80, 64, 40, BF, 8))
    y[::3] = 7
    truth = Truth(x, w, y, ignore=7)
    truth.check(*run(x, w, y, ignore_index=7))


@pytest.mark.parametrize("target", [-1, 900, 1 << 40, -(1 << 62)])
@pytest.mark.parametrize("columns", [0, 256])
def test_targets_outside(columns, target):
    """Such a token's loss and gradient are NaN, the other tokens' are theirs."""
    tokens, hidden, vocab = 90, 64, 900
    x, w, y = (t.cuda() for t in problem(tokens, hidden, vocab, BF, 9))
    more = dict(workspace=workspace(tokens, hidden, vocab, columns)) if columns else {}
    _, losses0, dx0, _ = run(x, w, y, **more)
    y[11] = target
    loss, losses, dx, dw = run(x, w, y, **more)
    keep = torch.arange(tokens, device="cuda") != 11
    assert bool(loss.isnan()) and bool(losses[11].isnan()) and bool(dx[11].isnan().all())
    assert bool(dw.isnan().all())
    assert torch.equal(losses[keep], losses0[keep]) and torch.equal(dx[keep], dx0[keep])


def test_not_finite_values():
    x, w, y = (t.cuda() for t in problem(70, 64, 800, BF, 10))
    _, losses0, dx0, _ = run(x, w, y)
    x[5, 3] = NAN
    loss, losses, dx, dw = run(x, w, y)
    keep = torch.arange(70, device="cuda") != 5
    assert bool(loss.isnan()) and bool(losses[5].isnan()) and bool(dw.isnan().all())
    assert torch.equal(losses[keep], losses0[keep]) and torch.equal(dx[keep], dx0[keep])
    # a word that no token can have: -inf logits everywhere
    x, w, y = (t.cuda() for t in problem(70, 64, 800, BF, 10))
    x[:, 0] = 1.0
    y[y == 300] = 301
    truth = Truth(x, torch.cat([w[:300], w[301:]]), y - (y > 300).long())
    w[300], w[300, 0] = 0.0, -float("inf")
    losses = torch.empty(70, device="cuda")
    loss = la.linear_cross_entropy(x, w, y, losses=losses)
    truth.check(loss, losses)


def test_what_is_not_wanted():
    x, w, y = (t.cuda() for t in problem(100, 128, 1000, BF, 11, 0.1))
    loss, losses, dx, dw = run(x, w, y)
    a = la.linear_cross_entropy_gradients(x, w, y, input_grad=False)
    b = la.linear_cross_entropy_gradients(x, w, y, weight_grad=False)
    assert a[1] is None and torch.equal(a[2], dw) and torch.equal(a[0], loss)
    assert b[2] is None and torch.equal(b[1], dx) and torch.equal(b[0], loss)
    out = torch.zeros(1, device="cuda")
    assert la.linear_cross_entropy(x, w, y, loss=out) is out and float(out) == float(loss)


def test_the_same_bits_again_and_on_another_stream():
    x, w, y = (t.cuda() for t in problem(500, 256, 3000, BF, 12, 0.1))
    first = run(x, w, y)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = run(x, w, y, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for p, q in zip(first, again):
        assert torch.equal(p, q)


def test_two_calls_at_once():
    """Two streams, a workspace each."""
    problems = [tuple(t.cuda() for t in problem(300, 192, 4000, BF, 20 + k, 0.1)) for k in (0, 1)]
    want = [run(*p) for p in problems]
    streams = [torch.cuda.Stream() for _ in problems]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [None, None]
    for _ in range(3):
        for k, s in enumerate(streams):
            got[k] = run(*problems[k], stream=s)
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for g, e in zip(got, want):
        for p, q in zip(g, e):
            assert torch.equal(p, q)


@pytest.mark.parametrize("columns", [0, 512])
def test_captured(columns):
    """Replays follow the inputs, the number of tokens that count among them."""
    tokens, hidden, vocab = 150, 128, 1500
    x, w, y = (t.cuda() for t in problem(tokens, hidden, vocab, BF, 13, 0.1))
    ws = workspace(tokens, hidden, vocab, columns)
    outs = dict(loss=torch.empty((), device="cuda"), losses=torch.empty(tokens, device="cuda"),
                dx=torch.empty_like(x), dweight=torch.empty_like(w))

    def step():
        la.linear_cross_entropy_gradients(x, w, y, workspace=ws, **outs)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k, ignored in enumerate((0.0, 0.9, 0.3, 1.1, 0.0)):
        for t, new in zip((x, w, y), problem(tokens, hidden, vocab, BF, 30 + k, ignored)):
            t.copy_(new)
        for t in outs.values():
            t.fill_(3)
        ws.fill_(255)  # what the workspace holds means nothing
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs.values()]
        fresh = workspace(tokens, hidden, vocab, columns)
        for p, q in zip(got, run(x, w, y, workspace=fresh)):
            assert torch.equal(p, q), k
        Truth(x, w, y).check(*got)


def test_piece_past_32_bits():
    """A held piece of more than 2^31 elements."""
    tokens, hidden, vocab = 16400, 64, 131200
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(tokens, hidden, device="cuda", generator=gen).to(BF)
    w = torch.randn(vocab, hidden, device="cuda", generator=gen).mul_(0.3).to(BF)
    y = torch.randint(0, vocab, (tokens,), device="cuda", generator=gen)
    ws = workspace(tokens, hidden, vocab, vocab)
    assert ws.numel() > 2 * (1 << 31)
    loss, losses, dx, dw = run(x, w, y, False, workspace=ws)
    rows = torch.tensor([0, 8000, tokens - 1], device="cuda")
    few = Truth(x[rows], w, y[rows], mean=False)
    few.check(None, losses[rows], dx[rows])
    # the last words' gradients, from all tokens' probabilities of them
    z = x.double() @ w[-3:].double().T
    lse = losses.double() + (x.double() * w[y].double()).sum(1)
    g = torch.exp(z - lse[:, None]) - (
        y[:, None] == torch.arange(vocab - 3, vocab, device="cuda")).double()
    want = g.T.contiguous() @ x.double()
    off = (dw[-3:].double() - want).abs()
    # as Truth counts it, lse being the kernel's own
    bound = (g.abs().T.contiguous() @ x.double().abs()) * (2.0 ** -8 * 1.01 + 2.0 ** -11 + U * 4096) \
        + 2.0 ** -8 * want.abs()
    assert bool((off <= bound).all()), float((off / bound).max())


@pytest.mark.parametrize("dtype", [BF, H])
def test_from_the_norm_to_the_step(dtype):
    """A model's end in training: final norm, projection and loss, back through
    both, and AdamW on their parameters from the gradients as they lie; against
    differentiation in 64 bits."""
    tokens, hidden, vocab, scale = 96, 256, 800, 256.0
    gen = torch.Generator().manual_seed(3)
    h = torch.randn(tokens, hidden, generator=gen).to(dtype).cuda()
    gamma = (1 + 0.1 * torch.randn(hidden, generator=gen)).to(dtype).cuda()
    w = (torch.randn(vocab, hidden, generator=gen) * 0.1).to(dtype).cuda()
    y = torch.randint(0, vocab, (tokens,), generator=gen).cuda()
    y[::5] = -100
    out, stats = la.rms_norm(h, gamma, eps=1e-6)
    loss, dout, dw = la.linear_cross_entropy_gradients(out, w, y, grad_scale=scale)
    dh, dgamma = la.rms_norm_backward(dout, h, gamma, stats)
    hd, gd, wd = (t.double().requires_grad_() for t in (h, gamma, w))
    od = hd * (hd.square().mean(1, keepdim=True) + 1e-6).rsqrt() * gd
    want_loss = torch.nn.functional.cross_entropy(od @ wd.T, y)
    want = torch.autograd.grad(scale * want_loss, (hd, gd, wd))
    # three tensors of 16 bits lie between a gradient and its inputs (out, g, dout), each
    # rounded by half a step at most, and the gradient itself: by the 2-norm, where the
    # roundings' sum enters through products that do not grow it, 4 halves
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -11
    for got, e in zip((dh, dgamma, dw), want):
        assert float((got.double() - e).norm() / e.norm()) < 4 * half
    # a rounded `out` moves each logit by at most half times the sum of its products' sizes
    moved = half * float((od.detach().abs() @ wd.detach().abs().T).max())
    assert abs(float(loss) - float(want_loss.detach())) < 2 * moved

    state = [(t.float(), torch.zeros(t.shape, device="cuda"), torch.zeros(t.shape, device="cuda"),
              t.clone()) for t in (gamma, w)]
    layer = la.Layer(state, [[dgamma], [dw]])
    found = torch.zeros(1, dtype=torch.int32, device="cuda")
    layer.check_gradients(found, grad_unscale=1.0 / scale)
    assert int(found) == 0
    before = [s[0].clone() for s in state]
    layer.step(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1,
               grad_unscale=1.0 / scale)
    for s, p, g in zip(state, before, (dgamma, dw)):
        g = g.double() / scale
        moved = (s[0] - p).double()
        # the first step from zero moments is lr along the gradient's signs
        assert float((moved + 1e-3 * g / (g.abs() + 1e-8)).abs().max()) <= \
            1e-3 * 2.0 ** -20 + float(p.abs().max()) * 2.0 ** -23
    # a target outside the vocabulary is an overflow to the check
    y[1] = vocab
    la.linear_cross_entropy_gradients(out, w, y, grad_scale=scale, dx=dout, dweight=dw)
    layer.check_gradients(found, grad_unscale=1.0 / scale)
    assert int(found) == 1
