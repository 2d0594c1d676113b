"""The Muon step on the GPU against its formula in 64 bits; the momentum bit
for bit against the same FP32 operations, the compute copy against the cast of
the GPU's own master."""
import pytest
import torch

import optimizer_step_layeradam_amd as la
from muonhelpers import DIRECTION, direction64, lr_factor, matrices, off

pytestmark = pytest.mark.gpu


def make(shapes, R, dtype, out, seed, grad_scale=1e-3):
    params, grads = [], []
    for i, s in enumerate(shapes):
        base = matrices(s, seed=seed + 10 * i, scale=grad_scale)
        grads.append([(base + matrices(s, seed=seed + 10 * i + 1 + r, scale=0.3 * grad_scale))
                      .to(dtype).cuda() for r in range(R)])
        params.append((matrices(s, seed=seed + 1000 + i, scale=0.02).cuda(),
                       matrices(s, seed=seed + 2000 + i, scale=2 * grad_scale).cuda(),
                       None if out is None else
                       torch.full(s, 7.0, dtype=out, device="cuda")))
    return params, grads


def reference(params, grads, lr, momentum=0.95, weight_decay=0.0, nesterov=True,
              grad_unscale=1.0, lr_scale="match_rms_adamw"):
    """Per tensor (master in 64 bits, momentum in 32, step times direction)."""
    out = []
    for (p, m, *_), gs in zip(params, grads):
        g = gs[0].float().cpu()
        for r in gs[1:]:
            g = g + r.float().cpu()
        mu = torch.tensor(momentum, dtype=torch.float32)
        g = g * torch.tensor(grad_unscale, dtype=torch.float32)
        m = mu * m.cpu() + g
        u = g + mu * m if nesterov else m
        s = lr * lr_factor(lr_scale, *p.shape[-2:])
        move = s * direction64(u)
        out.append((p.double().cpu() * (1.0 - lr * weight_decay) - move, m, move))
    return out


def check(params, ref):
    for (p, m, *w), (p64, m32, move) in zip(params, ref):
        assert torch.equal(m.cpu(), m32.view(m.shape))
        d = (p.double().cpu() - p64).flatten(-2).norm(dim=-1)
        # the direction's tolerance, and three roundings of the master's update
        bar = DIRECTION * move.flatten(-2).norm(dim=-1) + \
            3 * 2.0 ** -24 * (p64.flatten(-2).norm(dim=-1) + move.flatten(-2).norm(dim=-1))
        worst = float((d / bar.clamp(min=1e-300)).max())
        print(f"  {tuple(p.shape)}: {worst:.2f} of the bar", flush=True)
        assert worst <= 1.0
        if w and w[0] is not None:
            assert torch.equal(w[0].view(torch.int16), p.to(w[0].dtype).view(torch.int16))


SHAPES = [(1, 1), (1, 9), (9, 1), (64, 64), (127, 130), (130, 127), (300, 40), (40, 300),
          (3, 5, 9), (2, 33, 70), (2, 130, 100), (515, 257)]


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("R", [1, 2, 3, 8])
def test_layers(R, dtype, nesterov):
    out = {1: torch.bfloat16, 2: torch.float16, 3: None, 8: torch.bfloat16}[R]
    params, grads = make(SHAPES, R, dtype, out, seed=R)
    hp = dict(lr=1e-2, weight_decay=0.1, nesterov=nesterov, grad_unscale=1.0 / R)
    ref = reference(params, grads, **hp)
    la.muon_step(params, grads, **hp)
    check(params, ref)


@pytest.mark.parametrize("R", [4, 5, 6, 7])
def test_remaining_replica_counts(R):
    params, grads = make([(70, 90)], R, torch.bfloat16, torch.bfloat16, seed=40 + R)
    ref = reference(params, grads, lr=1e-3)
    la.muon_step(params, grads, lr=1e-3)
    check(params, ref)


@pytest.mark.parametrize("kind", sorted(la.LR_SCALES))
def test_scales_of_the_step(kind):
    params, grads = make([(200, 50), (50, 200), (2, 64, 64)], 1, torch.bfloat16, None, seed=60)
    ref = reference(params, grads, lr=1e-2, lr_scale=kind)
    la.muon_step(params, grads, lr=1e-2, lr_scale=kind)
    check(params, ref)


def test_three_steps_of_a_kept_layer():
    params, grads = make([(150, 260), (2, 90, 31)], 2, torch.bfloat16, torch.bfloat16, seed=70)
    layer = la.MuonLayer(params, grads)
    for k in range(3):
        ref = reference(params, grads, lr=1e-2, weight_decay=0.01, momentum=0.9)
        layer.step(lr=1e-2, weight_decay=0.01, momentum=0.9)
        check(params, ref)
        for gs in grads:
            for g in gs:
                g.copy_(matrices(tuple(g.shape), seed=80 + k, scale=1e-3))


def test_more_tensors_than_one_launch_takes():
    shapes = [(1 + 7 * i % 90, 1 + 17 * i % 110) for i in range(35)]
    params, grads = make(shapes, 2, torch.bfloat16, torch.bfloat16, seed=90)
    ref = reference(params, grads, lr=1e-2)
    la.muon_step(params, grads, lr=1e-2)
    check(params, ref)


def test_momentum_zero_and_lr_zero():
    params, grads = make([(60, 70)], 1, torch.bfloat16, torch.bfloat16, seed=95)
    before = params[0][0].clone()
    la.muon_step(params, grads, lr=0.0, momentum=0.0, weight_decay=0.1)
    assert torch.equal(params[0][0], before)
    assert torch.equal(params[0][1], grads[0][0].float())


def test_flag_and_nan_stay_with_their_matrix():
    params, grads = make([(3, 40, 50), (33, 20)], 2, torch.float16, torch.float16, seed=100)
    grads[0][1][1, 39, 49] = float("inf")
    ref = reference(params, grads, lr=1e-2)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    la.muon_step(params, grads, lr=1e-2, overflow_flag=flag)
    assert flag.item() == 1
    p, m, _ = params[0]
    assert torch.isnan(p[1]).all() and torch.isinf(m[1, 39, 49])
    check([tuple(x[::2] for x in params[0]), params[1]],
          [tuple(x[::2] for x in ref[0]), ref[1]])


def test_skip_leaves_everything_as_it_was():
    params, grads = make([(70, 90), (2, 20, 300)], 2, torch.bfloat16, torch.bfloat16, seed=110)
    keep = [[t.clone() for t in x] for x in params]
    layer = la.MuonLayer(params, grads,
                         torch.full((1 << 24,), 0xA5, dtype=torch.uint8, device="cuda"))
    assert layer.workspace_bytes() <= 1 << 24
    skip = torch.ones(1, dtype=torch.int32, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    grads[0][0][0, 0] = float("nan")
    layer.step(lr=1e-2, skip_if_nonzero=skip, overflow_flag=flag)
    for x, y in zip(params, keep):
        for a, b in zip(x, y):
            assert torch.equal(a, b)
    assert flag.item() == 0 and torch.all(layer._workspace == 0xA5)


def test_zero_gradient_of_a_zero_momentum():
    p, m = matrices((40, 30), seed=120).cuda(), torch.zeros(40, 30, device="cuda")
    before = p.clone()
    la.muon_step([(p, m)], [[torch.zeros(40, 30, dtype=torch.bfloat16, device="cuda")]],
                 lr=1e-2)
    assert torch.equal(p, before)


def test_whole_layer_with_adam_for_its_norms_in_one_graph():
    """As a training step uses them: one finite check for all gradients, the
    Muon step of the matrices and the AdamW step of the norm scales, both
    skipped on overflow, captured once and replayed."""
    params, grads = make([(96, 64), (64, 160), (160, 64)], 2, torch.float16, torch.float16,
                         seed=130)
    muon = la.MuonLayer(params, grads)
    n = 200
    norm = [(torch.ones(n, device="cuda"), torch.zeros(n, device="cuda"),
             torch.zeros(n, device="cuda"), torch.zeros(n, dtype=torch.float16, device="cuda"))]
    norm_grads = [[matrices((1, n), seed=140 + r, scale=1e-3).to(torch.float16).cuda()
                   for r in range(2)]]
    adam = la.Layer(norm, norm_grads)
    twin = [tuple(x.clone() for x in norm[0])]
    found = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = torch.ones(1, dtype=torch.int64, device="cuda")
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)

    def one_step():
        found.zero_()
        muon.check_gradients(found, grad_unscale=0.5)
        adam.check_gradients(found, grad_unscale=0.5)
        muon.step(lr=1e-3, weight_decay=0.01, grad_unscale=0.5, skip_if_nonzero=found)
        adam.step_ex(skip_if_nonzero=found, step_on_device=t, grad_unscale=0.5, **hp)
        t.add_((found == 0).to(torch.int64))

    def state():
        return [x.clone() for tup in (*params, *norm) for x in tup]

    for _ in range(2):
        ref = reference(params, grads, lr=1e-3, weight_decay=0.01, grad_unscale=0.5)
        one_step()  # eager, and the library's one-time reads before capture
        check(params, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one_step()
    other = torch.zeros(1 << 16, device="cuda")
    for k in range(4):
        overflow = k == 2
        held = grads[1][1][3, 3].clone()
        if overflow:
            grads[1][1][3, 3] = float("inf")
        ref = reference(params, grads, lr=1e-3, weight_decay=0.01, grad_unscale=0.5)
        before = state()
        graph.replay()
        other.add_(1.0)
        torch.cuda.synchronize()
        assert found.item() == int(overflow)
        if overflow:
            assert all(torch.equal(a, b) for a, b in zip(before, state()))
        else:
            check(params, ref)
        grads[1][1][3, 3] = held
    assert t.item() == 1 + 2 + 3
    for step in range(1, 6):
        la.step(twin, norm_grads, step=step, grad_unscale=0.5, **hp)
    assert torch.allclose(twin[0][0], norm[0][0], rtol=2.0 ** -22, atol=0)


def test_one_workspace_for_layers_in_turn():
    sets = [make(s, 1, torch.bfloat16, None, seed=150 + i)
            for i, s in enumerate(([(80, 200)], [(3, 90, 40), (10, 10)]))]
    layers = [la.MuonLayer(*x) for x in sets]
    ws = torch.empty(max(x.workspace_bytes() for x in layers), dtype=torch.uint8, device="cuda")
    layers = [la.MuonLayer(*x, workspace=ws) for x in sets]
    refs = [reference(*x, lr=1e-2) for x in sets]
    for x in layers:
        x.step(lr=1e-2)
    for x, ref in zip(sets, refs):
        check(x[0], ref)


def test_step_on_another_stream():
    params, grads = make([(200, 300)], 1, torch.bfloat16, torch.bfloat16, seed=160)
    ref = reference(params, grads, lr=1e-2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    la.muon_step(params, grads, lr=1e-2, stream=s)
    s.synchronize()
    check(params, ref)


def test_pinned_host_state():
    params, grads = make([(65, 130)], 1, torch.bfloat16, None, seed=170)
    ref = reference(params, grads, lr=1e-2)
    host = [tuple(torch.empty(t.shape, pin_memory=True).copy_(t) for t in params[0][:2])]
    la.muon_step(host, grads, lr=1e-2)
    torch.cuda.synchronize()
    check(host, ref)


def test_direction_is_what_orthogonalize_gives():
    params, grads = make([(2, 100, 140)], 1, torch.bfloat16, None, seed=180)
    u = params[0][1] * 0.95 + grads[0][0].float()
    o = la.orthogonalize(u, torch.empty_like(u, dtype=torch.float16))
    params[0][0].zero_()
    la.muon_step(params, grads, lr=1.0, lr_scale="none", nesterov=False)
    assert off(-params[0][0], o.double().cpu()) <= 2.0 ** -11
