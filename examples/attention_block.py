"""Trains one attention block over the points of a sphere on synthetic fields.

The block mixes all points: s <- s + dropout(attention(LN(s))), with the grid's
quadrature weights as the keys' weights, queries and keys normalised and turned by
colatitude and longitude.  It learns to match a teacher of the same kind.  Tokens are
channel-last rows [batch * points, channels]:

  forward   layer_norm_fwd, qk_norm_rope_fwd, attention_fwd, dropout_fwd (joins the stream)
  backward  dropout_bwd, attention_bwd, qk_norm_rope_bwd (both write into one buffer),
            layer_norm_bwd (adds the stream's gradient)
  update    muon_step for the projections, plain gradient steps for the vectors

Usage: python examples/attention_block.py [--steps N] [--channels C]
"""
import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import spherical_disco_convolution_amd as sdc  # noqa: E402


class Points:
    """Positions, frequencies and quadrature weights of an equiangular grid."""

    def __init__(self, nlat, nlon, pairs):
        theta = (torch.arange(nlat, device="cuda") + 0.5) * (math.pi / nlat)
        phi = torch.arange(nlon, device="cuda") * (2 * math.pi / nlon)
        self.count = nlat * nlon
        self.position = torch.stack((theta[:, None].expand(nlat, nlon), phi.expand(nlat, nlon)), dim=-1).reshape(-1, 2)
        # whole frequencies: periodic in longitude
        self.inv_freq = (torch.arange(pairs, device="cuda") % (pairs // 2) + 1).float()
        weight = torch.sin(theta)[:, None].expand(nlat, nlon).reshape(-1)
        self.log_weight = (weight / weight.sum()).log()


class Block:
    """Weights of the block and their gradients; `hq` query heads of `d`, `hkv` key heads."""

    def __init__(self, points, batch, channels, hq, hkv, d, p, dtype, gen):
        self.points, self.batch, self.hq, self.hkv, self.d, self.p, self.dtype = points, batch, hq, hkv, d, p, dtype

        def matrix(rows, cols):
            return torch.randn((rows, cols), generator=gen, device="cuda") / math.sqrt(rows)

        self.w = {"qkv": matrix(channels, (hq + 2 * hkv) * d), "out": matrix(hq * d, channels),
                  "gamma": torch.ones(channels, device="cuda"), "beta": torch.zeros(channels, device="cuda"),
                  "q": torch.ones(d, device="cuda"), "k": torch.ones(d, device="cuda")}
        self.momentum = {n: torch.zeros_like(self.w[n]) for n in ("qkv", "out")}
        self.bias = points.log_weight.repeat(batch)
        self.rope = dict(positions=points.position.repeat(batch, 1), inv_freq=points.inv_freq)

    def heads(self, qkv):
        """Queries, keys and values: columns of the projection's output."""
        hq, hkv, d = self.hq, self.hkv, self.d
        return (qkv[:, :hq * d].unflatten(1, (hq, d)), qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
                qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d)))

    def sequences(self, *tensors):
        return [t.unflatten(0, (self.batch, self.points.count)) for t in tensors]

    def forward(self, x, seed, offset):
        w = self.w
        y, _, mean, rstd = sdc.layer_norm_fwd(x, w["gamma"], w["beta"], axis=-1)
        qkv = y @ w["qkv"].to(self.dtype)
        q, k, v = self.heads(qkv)
        qn, kn = sdc.qk_norm_rope_fwd(q, k, w["q"], w["k"], **self.rope)
        o, lse = sdc.attention_fwd(*self.sequences(qn, kn, v), key_bias=self.bias)
        branch = o.view(x.shape[0], -1) @ w["out"].to(self.dtype)
        out = sdc.dropout_fwd(branch, self.p, seed, offset, residual=x)
        return out, (x, y, mean, rstd, qkv, qn, kn, o, lse, seed, offset)

    def backward(self, saved, gout):
        """Gradient of the input, and of the weights by name."""
        x, y, mean, rstd, qkv, qn, kn, o, lse, seed, offset = saved
        w, n = self.w, x.shape[0]
        g = {}
        gbranch = sdc.dropout_bwd(gout, self.p, seed, offset, gx_dtype=self.dtype)
        g["out"] = (o.view(n, -1).T @ gbranch).float()
        go = (gbranch @ w["out"].to(self.dtype).T).view(o.shape)
        q, k, v = self.heads(qkv)
        gqkv = torch.empty_like(qkv)
        gq, gk, gv = self.heads(gqkv)
        gqn, gkn, _ = sdc.attention_bwd(*self.sequences(qn, kn, v), o, lse, go, key_bias=self.bias,
                                        gv=self.sequences(gv)[0])
        _, _, g["q"], g["k"] = sdc.qk_norm_rope_bwd(q, k, gqn.flatten(0, 1), gkn.flatten(0, 1), w["q"], w["k"], gq=gq,
                                                    gk=gk, **self.rope)
        g["qkv"] = (y.T @ gqkv).float()
        gy = gqkv @ w["qkv"].to(self.dtype).T
        gx, g["gamma"], g["beta"] = sdc.layer_norm_bwd(x, gy, mean, rstd, w["gamma"], gsum=gout, axis=-1,
                                                       gx_dtype=self.dtype)
        return gx, g

    def update(self, g, lr):
        for n in ("qkv", "out"):
            sdc.muon_step(self.w[n], g[n], self.momentum[n], lr=lr)
        for n in ("gamma", "beta", "q", "k"):
            self.w[n] -= lr * g[n]


def train(steps=30, channels=128, nlat=17, nlon=32, batch=2, p=0.05, lr=0.05, seed=0, dtype=torch.bfloat16):
    """Losses of `steps` steps, mean squared error over all points and channels."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    points = Points(nlat, nlon, 16)
    teacher, student = (Block(points, batch, channels, 4, 2, 32, q, dtype, gen) for q in (0.0, p))
    losses = []
    for step in range(steps):
        x = torch.randn((batch * points.count, channels), generator=gen, device="cuda").to(dtype)
        target, _ = teacher.forward(x, seed, 0)
        out, saved = student.forward(x, seed, step)   # an offset of its own for every step
        diff = out.float() - target.float()
        losses.append(float(diff.square().mean()))
        _, g = student.backward(saved, (2.0 / diff.numel() * diff).to(dtype))
        student.update(g, lr * (1 - step / steps))
        print(f"step {step:3d}  loss {losses[-1]:.4f}", flush=True)
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--channels", type=int, default=128)
    a = ap.parse_args()
    train(a.steps, a.channels)
