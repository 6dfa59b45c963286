"""Float64 formulas of the attention, of the norm and rotation of its queries and
keys, and of dropout, with bounds on what rounding may do to them; shared by the
tests of these operators."""
import math

import numpy as np
import torch

F32, BF16 = torch.float32, torch.bfloat16
LOWEST = -1e30      # biases below leave a key out


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def sequences(cu_q, cu_k):
    return [(slice(a, b), slice(c, d)) for a, b, c, d in zip(cu_q[:-1], cu_q[1:], cu_k[:-1], cu_k[1:])]


def attention(q, k, v, bias, cu_q, cu_k, causal, scale, go=None, o_in=None, lse_in=None, dtype=BF16):
    """Values and bounds {name: (value, bound)} of o, lse and, with go, gq, gk, gv,
    on the CPU in float64.  q [T, Hq, dk], k [S, Hkv, dk], v [S, Hkv, dv]; tokens of
    no sequence hold NaN.  The bounds count, with u = 2^-24: products of dk, dv or n
    terms summed in float32 ((terms + 2) u of the sum of magnitudes), the exponent's
    argument and the exponential itself, and for bfloat16 half a step of each weight
    and each gradient of a score; results are off by half a step of their type."""
    u, half = 2.0 ** -24, half_step(dtype)
    low = half if dtype == BF16 else 0.0
    q, k, v = (t.double().cpu() for t in (q, k, v))
    tq, hq, dk = q.shape
    tk, hkv, dv = v.shape
    g = hq // hkv
    nan = float("nan")

    def make(*shape):
        return torch.full(shape, nan, dtype=torch.float64), torch.full(shape, nan, dtype=torch.float64)

    (o, eo), (lse, el) = make(tq, hq, dv), make(tq, hq)
    (gq, eq), (gk, ek), (gv, ev) = make(tq, hq, dk), make(tk, hkv, dk), make(tk, hkv, dv)
    for sq, sk in sequences(cu_q, cu_k):
        lq, lk = sq.stop - sq.start, sk.stop - sk.start
        seen = torch.ones(lq, lk, dtype=torch.bool)
        if causal:
            seen = torch.arange(lk)[None, :] <= torch.arange(lq)[:, None] + lk - lq
        b = torch.zeros(lk, dtype=torch.float64) if bias is None else bias.double().cpu()[sk]
        out = b < LOWEST
        seen = seen & ~out
        b = torch.where(out, 0.0, b)
        for t, e in ((gk, ek), (gv, ev)):
            t[sk], e[sk] = 0.0, 0.0
        for h in range(hq):
            qs = q[sq, h]
            ks, vs = (torch.where(out[:, None], 0.0, t[sk, h // g]) for t in (k, v))
            x = scale * qs @ ks.T + b
            ax = scale * qs.abs() @ ks.abs().T
            top = float(ax[seen].max()) if bool(seen.any()) else 0.0
            x = torch.where(seen, x, -math.inf)
            l = torch.logsumexp(x, 1) if lk else torch.full((lq,), -math.inf, dtype=torch.float64)
            lse[sq, h] = l
            big = float(l[l.isfinite()].abs().max()) if bool(l.isfinite().any()) else 0.0
            dx = (dk + 6) * u * top + 8 * u * (big + top + float(b.abs().max() if lk else 0.0))
            el[sq, h] = dx + (lk + 8) * u + 4 * u * l.abs().nan_to_num(posinf=0.0)
            dw = 2 * dx + (lk + 8) * u
            p = torch.exp(x - torch.where(l.isfinite(), l, 0.0)[:, None])
            o[sq, h] = p @ vs
            eo[sq, h] = (dw + low) * (p @ vs.abs()) + half * o[sq, h].abs()
            if go is None:
                continue
            gs, os = go.double().cpu()[sq, h], o_in.double().cpu()[sq, h]
            li = lse_in.double().cpu()[sq, h]
            p = torch.exp(x - torch.where(li.isfinite(), li, 0.0)[:, None])
            dp, delta = gs @ vs.T, (gs * os).sum(1, keepdim=True)
            err = (dv + 2) * u * (gs.abs() @ vs.abs().T + (gs * os).abs().sum(1, keepdim=True))
            ds = p * (dp - delta)
            es = p * (dw * (dp.abs() + delta.abs()) + err) + low * ds.abs()
            gq[sq, h] = scale * ds @ ks
            eq[sq, h] = scale * (es + (lk + 4) * u * ds.abs()) @ ks.abs()
            gk[sk, h // g] += scale * ds.T @ qs
            ek[sk, h // g] += scale * (es + (g * lq + 4) * u * ds.abs()).T @ qs.abs()
            gv[sk, h // g] += p.T @ gs
            ev[sk, h // g] += (p * (dw + low + (g * lq + 4) * u)).T @ gs.abs()
    res = {"o": (o, eo), "lse": (lse, el)}
    if go is not None:
        res.update(gq=(gq, eq + half * gq.abs()), gk=(gk, ek + half * gk.abs()), gv=(gv, ev + half * gv.abs()))
    return res


def check(name, got, want, bound, sizes=None):
    """got against want within bound wherever want is a number; -inf exactly."""
    got = got.double().cpu()
    part = ~want.isnan()
    inf = part & want.isinf()
    assert torch.equal(got[inf], want[inf]), name
    part &= ~inf
    far = (got - want).abs()[part] - bound[part]
    assert bool(got[part].isfinite().all()), f"{name}: not finite"
    assert far.numel() == 0 or float(far.max()) <= 1e-30, (
        f"{name}: {float(far.max()):.3g} over the bound; largest difference "
        f"{float((got - want).abs()[part].max()):.3g} of {float(want[part].abs().max()):.3g}")


def turns(positions, inv_freq, axes):
    """Angles [tokens, pairs] in float64."""
    pairs = inv_freq.numel()
    pos = positions.double().cpu().view(-1, axes)
    axis = torch.tensor([p * axes // pairs for p in range(pairs)], dtype=torch.long)
    return pos[:, axis] * inv_freq.double().cpu()


def rotate(x, angle, interleaved):
    """x [tokens, heads, d] turned by angle [tokens, pairs], pair by pair."""
    y = x.clone()
    pairs = angle.shape[1]
    for p in range(pairs):
        a, b = (2 * p, 2 * p + 1) if interleaved else (p, p + pairs)
        c, s = torch.cos(angle[:, p])[:, None], torch.sin(angle[:, p])[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
    return y


# ---------------------------------------------------------------------------
# Philox4x32 with ten rounds, in Python integers of 64 bits
# ---------------------------------------------------------------------------
def philox(c0, c1, c2, c3, k0, k1):
    """Words of counters given as uint64 arrays (below 2^32 each) under the key (k0, k1)."""
    m = np.uint64(0xffffffff)
    c0, c1, c2, c3 = (np.asarray(c, dtype=np.uint64) for c in (c0, c1, c2, c3))
    for r in range(10):
        a, b = c0 * np.uint64(0xD2511F53), c2 * np.uint64(0xCD9E8D57)
        r0, r1 = np.uint64((k0 + r * 0x9E3779B9) & 0xffffffff), np.uint64((k1 + r * 0xBB67AE85) & 0xffffffff)
        c0, c1, c2, c3 = (b >> np.uint64(32)) ^ c1 ^ r0, b & m, (a >> np.uint64(32)) ^ c3 ^ r1, a & m
    return c0, c1, c2, c3


def halves(n, seed, offset):
    """The half-words of elements 0 .. n - 1."""
    seed, offset = seed % 2 ** 64, offset % 2 ** 64
    blocks = np.arange((n + 7) // 8, dtype=np.uint64)
    lo, hi = blocks & np.uint64(0xffffffff), blocks >> np.uint64(32)
    words = philox(lo, hi, np.full_like(lo, offset & 0xffffffff), np.full_like(lo, offset >> 32), seed & 0xffffffff,
                   seed >> 32)
    out = np.stack([h for w in words for h in (w & np.uint64(0xffff), w >> np.uint64(16))], axis=1)
    return out.reshape(-1)[:n].astype(np.int64)
