"""Trains a small stack of pre-norm residual DISCO blocks on synthetic fields.

Each block is s <- s + DISCO(LN(s)); a last norm gives the output, which learns
to match a teacher: the same stack with other weights.  Fields and the layers'
weights are bfloat16, the optimiser's weights and momenta float32:

  forward   layer_norm_fwd (joins branch and residual stream), fused_fwd
  backward  fused_bwd, layer_norm_bwd (adds the stream's gradient)
  update    muon_step for the filters (it leaves the layer's bfloat16 copy),
            plain gradient steps for the norms' gamma and beta

Usage: python examples/train_block.py [--steps N] [--blocks L] [--channels C]
"""
import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import spherical_disco_convolution_amd as sdc  # noqa: E402


class Stack:
    """`blocks` residual blocks and a last norm, with their optimiser state."""

    def __init__(self, psi, blocks, channels, gen):
        self.psi = psi
        shape = (channels, channels, psi.K)
        # Psi holds quadrature weights, so a unit field comes out small: filters
        # are scaled to give a branch of about the stream's size, their updates too
        std = 1.0 / math.sqrt(channels * psi.K)
        probe = torch.randn((1, channels, psi.nlat_in, psi.nlon_in), generator=gen, device="cuda")
        w = std * torch.randn(shape, generator=gen, device="cuda")
        self.gain = 1.0 / float(sdc.fused_fwd(psi, probe, w).std())
        std *= self.gain
        self.w = [std * torch.randn(shape, generator=gen, device="cuda") for _ in range(blocks)]
        self.w16 = [w.to(torch.bfloat16) for w in self.w]
        self.momentum = [torch.zeros_like(w) for w in self.w]
        self.gamma = [torch.ones(channels, device="cuda") for _ in range(blocks + 1)]
        self.beta = [torch.zeros(channels, device="cuda") for _ in range(blocks + 1)]

    def forward(self, x):
        """Output of the stack and, per norm, what its gradient needs."""
        saved = []
        stream, branch = None, x
        for k in range(len(self.w) + 1):
            y, s, mean, rstd = sdc.layer_norm_fwd(branch, self.gamma[k], self.beta[k], residual=stream)
            stream = branch if s is None else s
            saved.append((y, stream, mean, rstd))
            if k < len(self.w):
                branch = sdc.fused_fwd(self.psi, y, self.w16[k], out_dtype=torch.bfloat16)
        return y, saved

    def backward(self, saved, gy):
        """Gradients of the filters, gammas and betas from the output's gradient."""
        n = len(self.w)
        gw, gg, gb = [None] * n, [None] * (n + 1), [None] * (n + 1)
        gs = None   # gradient that reaches the residual stream past the norm
        for k in range(n, -1, -1):
            _, s, mean, rstd = saved[k]
            gs, gg[k], gb[k] = sdc.layer_norm_bwd(s, gy, mean, rstd, self.gamma[k], gsum=gs,
                                                  gx_dtype=torch.bfloat16)
            if k > 0:   # gs is also the gradient of block k - 1's branch
                gy, gw[k - 1], _ = sdc.fused_bwd(self.psi, saved[k - 1][0], self.w16[k - 1], gs,
                                                 gx_dtype=torch.bfloat16)
        return gw, gg, gb

    def update(self, grads, lr):
        gw, gg, gb = grads
        for k, w in enumerate(self.w):
            sdc.muon_step(w, gw[k], self.momentum[k], lr=lr, weight_decay=0.01, scale=self.gain,
                          w16=self.w16[k])
        for k in range(len(self.gamma)):
            self.gamma[k] -= lr * gg[k]
            self.beta[k] -= lr * gb[k]


def train(steps=40, blocks=2, channels=64, nlat=33, nlon=64, batch=2, lr=0.1, seed=0):
    """Losses of `steps` steps, mean squared error over all points and channels."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    psi = sdc.psi_build(nlat, nlon, nlat, nlon, (3, 3), 4 * math.pi / (nlat - 1)).to_device()
    teacher, student = Stack(psi, blocks, channels, gen), Stack(psi, blocks, channels, gen)
    losses = []
    for step in range(steps):
        x = torch.randn((batch, channels, nlat, nlon), generator=gen, device="cuda").to(torch.bfloat16)
        target, _ = teacher.forward(x)
        out, saved = student.forward(x)
        diff = out.float() - target.float()
        losses.append(float(diff.square().mean()))
        gy = (2.0 / diff.numel() * diff).to(torch.bfloat16)
        # the momentum's scale drops out of the filters' update
        student.update(student.backward(saved, gy), lr * (1 - step / steps))
        print(f"step {step:3d}  loss {losses[-1]:.4f}", flush=True)
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--channels", type=int, default=64)
    a = ap.parse_args()
    train(a.steps, a.blocks, a.channels)
