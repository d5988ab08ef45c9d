"""A training step of residual blocks around the spherical convolution.

    h_0 = x;  u_i = norm(h_i) in 8 bits;  y_i = W_i . (F u_i);  h_{i+1} = h_i + y_i;  out = norm(h_n)
    loss = mean (out - target)^2 / 2

The blocks keep u_i as 8-bit values and scales (one byte a value where the contraction F u_i would take 2 K) and
h_i, the sum the norm stores; the backward reads u_i back, recomputes F u_i, and passes the rounding to 8 bits
straight through.  All gradients are clipped by their global norm before the update.

    python -m sparse_gather_contraction_amd.residual_step     # a few steps on one GPU, printing loss and norm
"""
from __future__ import annotations

import torch

from . import (disco_clip_grads, disco_dequantize, disco_fused_conv, disco_fused_conv_bwd, disco_rms_norm,
               disco_rms_norm_bwd, disco_rms_norm_f8)


class ResidualStack:
    """`blocks` blocks of `channels` channels over the filter `psi` (equal input and output grids), bf16 data and
    weights, fp32 norm weights."""

    def __init__(self, psi, channels: int, blocks: int, device="cuda", seed: int = 0):
        gen = torch.Generator(device=device).manual_seed(seed)
        std = 0.5 / (channels * psi.K) ** 0.5
        shape = (blocks, channels, channels, psi.K)
        self.psi = psi
        self.W = list((torch.randn(shape, generator=gen, device=device) * std).bfloat16().unbind(0))
        self.w = [torch.ones(channels, device=device) for _ in range(blocks + 1)]

    def parameters(self):
        return self.W + self.w

    def forward(self, x):
        """(out, what the backward needs): per block (q, scale) of u and the sum h; the last sum."""
        kept, y, h = [], x, None
        for W, w in zip(self.W, self.w):
            if h is None:  # the first block's sum is x itself
                q, scale = disco_rms_norm_f8(y, w)
                h = x
            else:
                q, scale, h = disco_rms_norm_f8(y, w, residual=h)
            kept.append((q, scale, h))
            y = disco_fused_conv(self.psi, disco_dequantize(q, scale, dtype=x.dtype), W)
        if h is None:
            return disco_rms_norm(x, self.w[0]), (kept, x)
        out, h = disco_rms_norm(y, self.w[-1], residual=h)
        return out, (kept, h)

    def backward(self, saved, gout):
        """The gradients of the parameters, in their order, and of x."""
        kept, h = saved
        dW, dw = [None] * len(self.W), [None] * len(self.w)
        gh, dw[-1] = disco_rms_norm_bwd(h, self.w[-1], gout)
        for i in reversed(range(len(self.W))):
            q, scale, h = kept[i]
            gu, dW[i] = disco_fused_conv_bwd(self.psi, disco_dequantize(q, scale, dtype=gh.dtype), self.W[i], gh)
            gh, dw[i] = disco_rms_norm_bwd(h, self.w[i], gu, gh=gh)
        return dW + dw, gh

    def step(self, x, target, lr: float, max_norm: float = 1.0):
        """One step of gradient descent; (loss, the gradients' norm before clipping), both on the device."""
        out, saved = self.forward(x)
        diff = out.float() - target
        grads, _ = self.backward(saved, (diff / diff.numel()).to(out.dtype))
        norm = disco_clip_grads(grads, max_norm)
        for p, g in zip(self.parameters(), grads):
            p.add_(g, alpha=-lr)
        return diff.square().mean() / 2, norm


def main(steps: int = 8):
    from disco_inputs.psi import build_psi

    from . import disco_psi_create

    psi = disco_psi_create(build_psi(64, 128, 64, 128, 0.15, 3, 3))
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, target = (torch.randn((2, 64, 64, 128), generator=gen, device="cuda") for _ in range(2))
    model = ResidualStack(psi, 64, 3)
    for i in range(steps):
        loss, norm = model.step(x.bfloat16(), target, lr=1.0)
        print(f"step {i}: loss {float(loss):.6f}, gradient norm {float(norm):.6f}", flush=True)


if __name__ == "__main__":
    main()
