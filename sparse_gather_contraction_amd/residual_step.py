"""A training step of residual blocks around the spherical convolution.

    h_0 = x;  u_i = norm(h_i) in 8 bits;  y_i = W_i . (F u_i);  h_{i+1} = h_i + y_i;  out = norm(h_n)
    loss = mean (out - target)^2 / 2

The blocks keep u_i as 8-bit values and scales (one byte a value where the contraction F u_i would take 2 K) and
h_i, the sum the norm stores; the backward reads u_i back, recomputes F u_i, and passes the rounding to 8 bits
straight through.  All gradients are clipped by their global norm before the update.

With `hidden` channels each block is followed by a pointwise one, its products in 8-bit integers:

    v_i = norm(h) in int8;  a_i = V1_i v_i + c1_i;  g_i = gelu(a_i) in int8;  y_i = V2_i g_i + c2_i;  h <- h + y_i

It keeps v_i, g_i (the products' operands) and a_i, one byte a value each, with a scale for each point; the backward's
products read them as they are, and gelu's slope is taken at the kept a_i.

    python -m sparse_gather_contraction_amd.residual_step [hidden]   # a few steps on one GPU, printing loss and norm
"""
from __future__ import annotations

import sys

import torch

from . import (disco_clip_grads, disco_dequantize, disco_fused_conv, disco_fused_conv_bwd, disco_linear_i8,
               disco_linear_i8_bwd_input, disco_linear_i8_bwd_weight, disco_quantize_i8, disco_rms_norm,
               disco_rms_norm_bwd, disco_rms_norm_f8)


class ResidualStack:
    """`blocks` blocks of `channels` channels over the filter `psi` (equal input and output grids), each followed by a
    pointwise one of `hidden` channels (0: none), bf16 data and weights, fp32 norm weights and biases."""

    def __init__(self, psi, channels: int, blocks: int, device="cuda", seed: int = 0, hidden: int = 0):
        gen = torch.Generator(device=device).manual_seed(seed)
        std = 0.5 / (channels * psi.K) ** 0.5
        shape = (blocks, channels, channels, psi.K)
        self.psi = psi
        self.W = list((torch.randn(shape, generator=gen, device=device) * std).bfloat16().unbind(0))
        self.w = [torch.ones(channels, device=device) for _ in range(blocks + 1)]
        self.pointwise = []
        for _ in range(blocks if hidden else 0):
            V1 = (torch.randn((hidden, channels), generator=gen, device=device) * 0.5 / channels ** 0.5).bfloat16()
            V2 = (torch.randn((channels, hidden), generator=gen, device=device) * 0.5 / hidden ** 0.5).bfloat16()
            self.pointwise.append([V1, torch.zeros(hidden, device=device), V2, torch.zeros(channels, device=device),
                                   torch.ones(channels, device=device)])

    def parameters(self):
        return self.W + self.w + [p for block in self.pointwise for p in block]

    def _pointwise_forward(self, block, y, h):
        """(y, the sum h, what the backward needs) of one pointwise block on h + y."""
        V1, c1, V2, c2, w = block
        v, h = disco_rms_norm(y, w, residual=h)
        W1, W2 = disco_quantize_i8(V1), disco_quantize_i8(V2)
        u = disco_quantize_i8(v)
        a = disco_linear_i8(*u, *W1, bias=c1, dtype=y.dtype)
        g, gs, a8, a8s = disco_quantize_i8(a, act="gelu", keep=True)
        y = disco_linear_i8(g, gs, *W2, bias=c2, dtype=y.dtype)
        return y, h, (u, (g, gs), (a8, a8s), W1, W2, h)

    def _pointwise_backward(self, block, kept, gh):
        """The gradients of the block's parameters, and of the sum it was given."""
        V1, _, V2, _, w = block
        u, g, a8, W1, W2, h = kept
        dV2, dc2 = disco_linear_i8_bwd_weight(gh, *g, channels=V2.shape[1], bias=True)
        ga = disco_linear_i8_bwd_input(gh, *W2, channels=V2.shape[1], act="gelu", kept=a8[0], kept_scale=a8[1])
        dV1, dc1 = disco_linear_i8_bwd_weight(ga, *u, channels=V1.shape[1], bias=True)
        gv = disco_linear_i8_bwd_input(ga, *W1, channels=V1.shape[1])
        gh, dw = disco_rms_norm_bwd(h, w, gv, gh=gh)
        return [dV1, dc1, dV2, dc2, dw], gh

    def forward(self, x):
        """(out, what the backward needs): per block (q, scale) of u and the sum h; the last sum; the pointwise blocks'."""
        kept, points, y, h = [], [], x, None
        for i, (W, w) in enumerate(zip(self.W, self.w)):
            if h is None:  # the first block's sum is x itself
                q, scale = disco_rms_norm_f8(y, w)
                h = x
            else:
                q, scale, h = disco_rms_norm_f8(y, w, residual=h)
            kept.append((q, scale, h))
            y = disco_fused_conv(self.psi, disco_dequantize(q, scale, dtype=x.dtype), W)
            if self.pointwise:
                y, h, p = self._pointwise_forward(self.pointwise[i], y, h)
                points.append(p)
        if h is None:
            return disco_rms_norm(x, self.w[0]), (kept, x, points)
        out, h = disco_rms_norm(y, self.w[-1], residual=h)
        return out, (kept, h, points)

    def backward(self, saved, gout):
        """The gradients of the parameters, in their order, and of x."""
        kept, h, points = saved
        dp = [None] * len(points)
        dW, dw = [None] * len(self.W), [None] * len(self.w)
        gh, dw[-1] = disco_rms_norm_bwd(h, self.w[-1], gout)
        for i in reversed(range(len(self.W))):
            if points:
                dp[i], gh = self._pointwise_backward(self.pointwise[i], points[i], gh)
            q, scale, h = kept[i]
            gu, dW[i] = disco_fused_conv_bwd(self.psi, disco_dequantize(q, scale, dtype=gh.dtype), self.W[i], gh)
            gh, dw[i] = disco_rms_norm_bwd(h, self.w[i], gu, gh=gh)
        return dW + dw + [g for block in dp for g in block], gh

    def step(self, x, target, lr: float, max_norm: float = 1.0):
        """One step of gradient descent; (loss, the gradients' norm before clipping), both on the device."""
        out, saved = self.forward(x)
        diff = out.float() - target
        grads, _ = self.backward(saved, (diff / diff.numel()).to(out.dtype))
        norm = disco_clip_grads(grads, max_norm)
        for p, g in zip(self.parameters(), grads):
            p.add_(g, alpha=-lr)
        return diff.square().mean() / 2, norm


def main(steps: int = 8, hidden: int = 0):
    from disco_inputs.psi import build_psi

    from . import disco_psi_create

    psi = disco_psi_create(build_psi(64, 128, 64, 128, 0.15, 3, 3))
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, target = (torch.randn((2, 64, 64, 128), generator=gen, device="cuda") for _ in range(2))
    model = ResidualStack(psi, 64, 3, hidden=hidden)
    for i in range(steps):
        loss, norm = model.step(x.bfloat16(), target, lr=1.0)
        print(f"step {i}: loss {float(loss):.6f}, gradient norm {float(norm):.6f}", flush=True)


if __name__ == "__main__":
    main(hidden=int(sys.argv[1]) if len(sys.argv) > 1 else 0)
