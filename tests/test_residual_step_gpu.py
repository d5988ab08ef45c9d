"""The training step of residual blocks (norm in 8 bits, its reader, the convolution, the norms' backward, clipping)
against the same step in fp64 with the filter as a dense array and autograd's gradients.

The reference takes the step's own 8-bit values (their rounding is passed straight through), so what is left are the
bf16 roundings between the stages.  From the loss to a gradient of two blocks there are fewer than ten of them in a
row (out, its gradient, per block: the sum, F u, y, the gradients of F u, u and the sum), each at most 2^-8 of its
value, so a gradient's relative L2 distance is below 10 x 2^-8."""
import pytest
import torch

import sparse_gather_contraction_amd as sgc
from disco_inputs.psi import build_psi
from sparse_gather_contraction_amd.residual_step import ResidualStack

pytestmark = pytest.mark.gpu

H, W, C, BLOCKS = 16, 32, 16, 2


def make():
    csr = build_psi(H, W, H, W, 0.5, 2, 2)
    return csr, ResidualStack(sgc.disco_psi_create(csr, 0), C, BLOCKS, seed=3)


def dense(csr):
    F = torch.zeros((csr.K, H, H, W), dtype=torch.float64)  # [basis, output latitude, input latitude, longitude offset]
    for row in range(csr.K * H):
        for e in range(int(csr.row_ptr[row]), int(csr.row_ptr[row + 1])):
            F[row // H, row % H, int(csr.col_hi[e]), int(csr.col_wi[e])] += float(csr.val[e])
    return F


def norm(h, w):
    return h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w.view(1, -1, 1, 1)


def inputs():
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, target = (torch.randn((2, C, H, W), generator=gen, device="cuda") for _ in range(2))
    return x.bfloat16(), target


def test_gradients_against_autograd_in_fp64():
    csr, model = make()
    x, target = inputs()
    out, saved = model.forward(x)
    diff = out.float() - target
    grads, gx = model.backward(saved, (diff / diff.numel()).to(out.dtype))
    F = dense(csr)
    at = (torch.arange(W).view(1, -1) + torch.arange(W).view(-1, 1)) % W  # [wo, offset] -> input longitude
    leaf = [p.detach().double().cpu().requires_grad_() for p in model.parameters()]
    X = x.double().cpu().requires_grad_()
    h, y = X, None
    for i, (q, scale, _) in enumerate(saved[0]):
        h = X if y is None else h + y
        u = norm(h, leaf[BLOCKS + i])
        kept = sgc.disco_dequantize(q, scale).double().cpu()
        assert float((kept - u.detach()).norm() / u.detach().norm()) <= 2.0 ** -4 + 10 * 2.0 ** -8  # 8 bits: 2^-4 a value
        u = u + (kept - u).detach()
        Fu = torch.einsum("kpij,bcioj->bckpo", F, u[..., at])
        y = torch.einsum("ock,bckpw->bopw", leaf[i], Fu)
    ref = norm(h + y, leaf[-1])
    assert float((out.double().cpu() - ref.detach()).norm() / ref.detach().norm()) <= 10 * 2.0 ** -8
    ((ref - target.double().cpu()).square().mean() / 2).backward()
    for name, got, want in [(f"parameter {i}", g, p.grad) for i, (g, p) in enumerate(zip(grads, leaf))] + [("x", gx, X.grad)]:
        err = float((got.double().cpu() - want).norm() / want.norm())
        assert err <= 10 * 2.0 ** -8, (name, err)


def test_step_clips_and_descends():
    _, model = make()
    x, target = inputs()
    before = [p.clone() for p in model.parameters()]
    out, saved = model.forward(x)
    diff = out.float() - target
    grads, _ = model.backward(saved, (diff / diff.numel()).to(out.dtype))
    ref = sum(float(g.double().square().sum()) for g in grads) ** 0.5
    first, norm0 = model.step(x, target, lr=0.5, max_norm=ref / 2)
    assert abs(float(norm0) - ref) <= 2.0 ** -23 * ref
    for p, b, g in zip(model.parameters(), before, grads):
        # the clipped gradient and the weight's new value are rounded once each
        step = g.double() * (0.5 * (ref / 2) / (ref + 1e-6))
        eps = torch.finfo(p.dtype).eps / 2
        assert bool(((p.double() - (b.double() - step)).abs() <= eps * 1.01 * (step.abs() + p.double().abs()) + 2.0 ** -40).all())
    for _ in range(6):
        last, _ = model.step(x, target, lr=0.5, max_norm=1.0)
    assert float(last) < float(first)
