"""The training step of residual blocks with pointwise blocks between them (products in 8-bit integers, gelu's checkpoint in
8 bits) against the same step in fp64 with autograd's gradients.

The reference takes the step's own 8-bit values, whose rounding is passed straight through, and gelu's slope at the kept
values.  What is left are roundings to bf16, each at most 2^-8 of its value: from the loss to a gradient fewer than ten in a
row for the two convolution blocks, and for each pointwise block eight more (v, a, y, both weights and gradients, the operand
of a weight's gradient): 26 x 2^-8."""
import pytest
import torch

import sparse_gather_contraction_amd as sgc
from disco_inputs.psi import build_psi
from sparse_gather_contraction_amd.residual_step import ResidualStack
from test_residual_step_gpu import BLOCKS, C, H, W, dense, inputs, norm

pytestmark = pytest.mark.gpu

HIDDEN = 40   # no multiple of 16
TOL = 26 * 2.0 ** -8


def make():
    csr = build_psi(H, W, H, W, 0.5, 2, 2)
    model = ResidualStack(sgc.disco_psi_create(csr, 0), C, BLOCKS, seed=3, hidden=HIDDEN)
    gen = torch.Generator(device="cuda").manual_seed(9)
    for block in model.pointwise:  # biases that matter
        for p in (block[1], block[3]):
            p.add_(torch.randn(p.shape, generator=gen, device="cuda") * 0.3)
    return csr, model


def values(q, scale, channels):
    """A form's values as a field in fp64, read apart from the library."""
    return (q.double() * scale.double().unsqueeze(-1))[..., :channels].movedim(-1, 1).cpu()


def through(exact, held):
    """`held` in the forward, exact's gradient."""
    return exact + (held - exact).detach()


def test_gradients_against_autograd_in_fp64():
    csr, model = make()
    x, target = inputs()
    out, saved = model.forward(x)
    diff = out.float() - target
    grads, gx = model.backward(saved, (diff / diff.numel()).to(out.dtype))
    params = model.parameters()
    assert [g.shape for g in grads] == [p.shape for p in params]
    F = dense(csr)
    at = (torch.arange(W).view(1, -1) + torch.arange(W).view(-1, 1)) % W
    leaf = [p.detach().double().cpu().requires_grad_() for p in params]
    conv, norms, points = leaf[:BLOCKS], leaf[BLOCKS:2 * BLOCKS + 1], leaf[2 * BLOCKS + 1:]
    X = x.double().cpu().requires_grad_()
    h, y = X, None
    for i, (q, scale, _) in enumerate(saved[0]):
        h = X if y is None else h + y
        u = norm(h, norms[i])
        u = through(u, sgc.disco_dequantize(q, scale).double().cpu())
        y = torch.einsum("ock,bckpw->bopw", conv[i], torch.einsum("kpij,bcioj->bckpo", F, u[..., at]))
        V1, c1, V2, c2, w = points[5 * i:5 * i + 5]
        u8, g8, a8, W1, W2, _ = saved[2][i]
        h = h + y
        v = norm(h, w)
        held = values(*u8, C)
        assert float((held - v.detach()).norm() / v.detach().norm()) <= 0.02 + TOL  # 8 bits of the largest value
        v = through(v, held)
        a = torch.einsum("oc,bchw->bohw", through(V1, values(*W1, C)), v) + c1.view(1, -1, 1, 1)
        ak = values(*a8, HIDDEN)
        assert float((ak - a.detach()).norm() / a.detach().norm()) <= 0.02 + TOL
        slope = torch.special.ndtr(ak) + ak * torch.exp(-ak * ak / 2) / (2 * torch.pi) ** 0.5
        g = values(*g8, HIDDEN) + slope * (a - a.detach())
        y = torch.einsum("oc,bchw->bohw", through(V2, values(*W2, HIDDEN)), g) + c2.view(1, -1, 1, 1)
    ref = norm(h + y, norms[-1])
    assert float((out.double().cpu() - ref.detach()).norm() / ref.detach().norm()) <= TOL
    ((ref - target.double().cpu()).square().mean() / 2).backward()
    for name, got, want in [(f"parameter {i}", g, p.grad) for i, (g, p) in enumerate(zip(grads, leaf))] + [("x", gx, X.grad)]:
        err = float((got.double().cpu() - want).norm() / want.norm())
        assert err <= TOL, (name, err)


def test_steps_run():
    _, model = make()
    x, target = inputs()
    before = [p.clone() for p in model.parameters()]
    for _ in range(3):
        loss, gnorm = model.step(x, target, lr=0.1)
        assert bool(torch.isfinite(loss)) and bool(torch.isfinite(gnorm)) and float(gnorm) > 0
    assert all(not torch.equal(p, b) for p, b in zip(model.parameters(), before))


def test_a_step_is_reproducible_and_replayed():
    _, model = make()
    x, target = inputs()
    out, saved = model.forward(x)
    gout = ((out.float() - target) / target.numel()).to(out.dtype)
    grads, gx = model.backward(saved, gout)
    again, _ = model.backward(model.forward(x)[1], gout)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        model.backward(model.forward(x)[1], gout)  # everything is loaded before the capture
    side.synchronize()
    with torch.cuda.graph(graph, stream=side):
        out2, saved2 = model.forward(x)
        grads2, gx2 = model.backward(saved2, gout)
    for k in range(3):
        x.copy_(inputs()[0] * (1 + k))
        eager_out, eager_saved = model.forward(x)
        eager, eager_gx = model.backward(eager_saved, gout)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out2, eager_out) and torch.equal(gx2, eager_gx)
        assert all(torch.equal(a, b) for a, b in zip(grads2, eager))
