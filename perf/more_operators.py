"""Workloads of the attention over points, of the norm and rotation of its queries and keys, and of dropout.

`run` with ``own`` false computes them in elementary float32 torch operations
(angles in float64); with ``own`` true through the package's entry points.
`exact` is float64.
"""
import math
import random

import torch

own = False

F32, BF16 = "f32", "bf16"
DTYPES = {F32: torch.float32, BF16: torch.bfloat16}
QK_EPS = 1e-6
CHUNK = 1 << 28          # elements of a score matrix held at once


def listed():
    return [
        # a 9 x 17 field, two heads: one launch's latency
        dict(name="attn_fwd_tiny_f32", op="attn_fwd", mode="grid", seqs=1, q=153, k=153, hq=2, hkv=2, dk=32, dv=32,
             dtype=F32, bias=True, causal=False),
        # eight points sampled from a 129 x 256 field: few queries, many keys
        dict(name="attn_fwd_points8_bf16", op="attn_fwd", mode="grid", seqs=1, q=8, k=33024, hq=16, hkv=2, dk=128,
             dv=128, dtype=BF16, bias=True, causal=False),
        # time series of different lengths in one batch, each step sees the ones before it
        dict(name="attn_fwd_packed_bf16", op="attn_fwd", mode="packed", seqs=9, q=12001, k=12001, hq=12, hkv=4, dk=128,
             dv=128, dtype=BF16, bias=False, causal=True),
        # global attention over the 129 x 256 field, quadrature weights on the keys
        dict(name="attn_fwd_c2_bf16", op="attn_fwd", mode="grid", seqs=1, q=33024, k=33024, hq=8, hkv=8, dk=64, dv=64,
             dtype=BF16, bias=True, causal=False),
        # training in float32 on two 33 x 64 fields
        dict(name="attn_bwd_c1_f32", op="attn_bwd", mode="grid", seqs=2, q=4224, k=4224, hq=4, hkv=4, dk=32, dv=32,
             dtype=F32, bias=True, causal=False),
        # training on the packed series
        dict(name="attn_bwd_packed_bf16", op="attn_bwd", mode="packed", seqs=7, q=6007, k=6007, hq=12, hkv=4, dk=128,
             dv=128, dtype=BF16, bias=False, causal=True),
        # training on a 65 x 128 field
        dict(name="attn_bwd_grid_bf16", op="attn_bwd", mode="grid", seqs=1, q=8320, k=8320, hq=8, hkv=8, dk=64, dv=64,
             dtype=BF16, bias=True, causal=False),
        # the sampler's eight points
        dict(name="qk_fwd_rows8_bf16", op="qk_fwd", tokens=8, hq=16, hkv=2, d=128, rot=128, axes=1, interleaved=False,
             dtype=BF16),
        # every point of the 129 x 256 field, turned by colatitude and longitude over half of each head
        dict(name="qk_fwd_c2_bf16", op="qk_fwd", tokens=33024, hq=12, hkv=4, d=128, rot=64, axes=2, interleaved=False,
             dtype=BF16),
        # its gradient, pairs side by side
        dict(name="qk_bwd_c2_bf16", op="qk_bwd", tokens=33024, hq=12, hkv=4, d=128, rot=128, axes=1, interleaved=True,
             dtype=BF16),
        # the 0.25 degree layer's branch joined to the residual stream
        dict(name="drop_fwd_c4_bf16_res", op="drop_fwd", outer=128, inner=721 * 1440, p=0.1, x=BF16, y=BF16,
             residual=True),
        # training on channel-last rows of odd width
        dict(name="drop_bwd_rows_f32", op="drop_bwd", outer=16383, inner=2047, p=0.25, x=F32, y=F32, residual=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_fwd", "attn_bwd", "attn_bwd", "qk_fwd", "qk_bwd", "drop_fwd", "drop_bwd"])
    dtype = rng.choice([F32, BF16, BF16])
    if op in ("attn_fwd", "attn_bwd"):
        hkv = rng.choice([1, 2, 3, 4, 8])
        hq = hkv * rng.choice([1, 1, 2, 3, 4, 8])
        dk = rng.choice([16, 24, 32, 40, 64, 64, 96, 128, 128])
        dv = dk if rng.random() < 0.7 else rng.choice([16, 32, 64, 128])
        mode = rng.choice(["grid", "grid", "points", "packed"])
        if mode == "points":
            seqs = rng.randint(1, 4)
            q, k = seqs * rng.randint(1, 64), seqs * _log_int(rng, 100, 33024)
        elif mode == "grid":
            seqs = rng.randint(1, 4)
            q = k = seqs * _log_int(rng, 45, 33024)
        else:
            seqs = rng.randint(2, 24)
            q = k = _log_int(rng, 8 * seqs, 16384)
        case = dict(op=op, mode="packed" if mode == "packed" else "grid", seqs=seqs, q=q, k=k, hq=hq, hkv=hkv, dk=dk,
                    dv=dv, dtype=dtype, bias=rng.random() < 0.5,
                    causal=mode == "packed" or (mode == "grid" and rng.random() < 0.2))
        # float32 products take sixteen times as long as bfloat16 ones
        most = (5e11 if op == "attn_fwd" else 4e11) * (0.1 if dtype == F32 else 1.0)
        while work(case)["flops"] > most:
            case["k"] = max(seqs * 40, (case["k"] // seqs) * 3 // 4 * seqs)
            case["q"] = min(case["q"], case["k"]) if mode == "points" else case["k"]
        return case
    if op in ("qk_fwd", "qk_bwd"):
        hkv = rng.choice([1, 2, 4, 8])
        d = rng.choice([16, 32, 40, 64, 96, 128, 256])
        axes = rng.choice([1, 1, 2])
        tokens, hq = _log_int(rng, 1, 33024), hkv * rng.choice([1, 2, 3, 4])
        while tokens * (hq + hkv) * d > 33024 * 16 * 128:
            tokens = max(1, tokens // 2)
        return dict(op=op, tokens=tokens, hq=hq, hkv=hkv, d=d, rot=d if rng.random() < 0.5 else d // 8 * 4, axes=axes,
                    interleaved=rng.random() < 0.5, dtype=dtype)
    outer, inner = _log_int(rng, 1, 16384), _log_int(rng, 1, 1 << 20)
    while outer * inner > 1 << 26:
        outer = max(1, outer // 2)
    y = rng.choice([F32, BF16])
    return dict(op=op, outer=outer, inner=inner, p=rng.choice([0.0, 0.05, 0.1, 0.25, 0.5, 0.9]), x=dtype, y=y,
                residual=op == "drop_fwd" and rng.random() < 0.6)


def _lengths(case):
    """Queries and keys of each sequence: equal shares, or a few long ones among many short ones."""
    n, total = case["seqs"], case["q"]
    if case["mode"] == "grid":
        return [case["q"] // n] * n, [case["k"] // n] * n
    rng = random.Random(1000003 * n + total)
    share = [rng.random() ** 3 + 0.01 for _ in range(n)]
    lens = [max(1, int(total * s / sum(share))) for s in share]
    lens[0] = 1                                      # a series that has just begun
    lens[-1] += total - sum(lens)
    return lens, lens


def _normal(gen, shape, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    st = {"case": dict(case)}
    if case["op"] in ("attn_fwd", "attn_bwd"):
        tq, tk, hq, hkv, dk, dv = (case[n] for n in ("q", "k", "hq", "hkv", "dk", "dv"))
        dt = DTYPES[case["dtype"]]
        # keys and values of one projection, side by side; scores of spread two, as trained heads have
        st["q"] = (2.0 * _normal(gen, (tq, hq, dk))).to(dt)
        kv = _normal(gen, (tk, hkv * (dk + dv)), dt)
        st["k"] = kv[:, :hkv * dk].unflatten(1, (hkv, dk))
        st["v"] = kv[:, hkv * dk:].unflatten(1, (hkv, dv))
        lq, lk = _lengths(case)
        if case["mode"] == "packed":
            st["cu"] = torch.tensor([sum(lq[:i]) for i in range(len(lq) + 1)], dtype=torch.int32, device="cuda")
        st["bias"] = None
        if case["bias"]:
            # logarithms of quadrature weights from pole to pole; a twentieth of the points is masked out
            w = torch.cat([torch.sin((torch.arange(n, device="cuda", dtype=torch.float32) + 0.5) * (math.pi / n)).log()
                           for n in lk])
            st["bias"] = torch.where(torch.rand(w.shape, generator=gen, device="cuda") < 0.05, -math.inf, w)
        if case["op"] == "attn_bwd":
            o, st["lse"] = _attn_fwd_plain(st)
            st["o"] = o
            st["go"] = _normal(gen, (tq, hq, dv), dt)
        return st
    if case["op"] in ("qk_fwd", "qk_bwd"):
        t, hq, hkv, d, rot, dt = case["tokens"], case["hq"], case["hkv"], case["d"], case["rot"], DTYPES[case["dtype"]]
        # the projection's output: queries, keys and values of a token side by side
        qkv = _normal(gen, (t, (hq + 2 * hkv) * d), dt)
        st["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        st["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        st["qw"], st["kw"] = 1.0 + 0.1 * _normal(gen, (d,)), 1.0 + 0.1 * _normal(gen, (d,))
        if case["axes"] == 2:      # colatitude and longitude, whole frequencies: periodic in longitude
            u = torch.rand((t, 2), generator=gen, device="cuda")
            st["pos"] = u * torch.tensor([math.pi, 2 * math.pi], device="cuda")
            st["freq"] = (torch.arange(rot // 2, device="cuda") % max(1, rot // 4) + 1).float()
        else:                      # steps of a series far from its beginning
            first = int(torch.randint(0, 1 << 20, (1,), generator=gen, device="cuda"))
            st["pos"] = first + torch.arange(t, dtype=torch.int32, device="cuda")
            st["freq"] = (10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)).float()
        if case["op"] == "qk_bwd":
            st["gq"], st["gk"] = _normal(gen, (t, hq, d), dt), _normal(gen, (t, hkv, d), dt)
        return st
    shape = (case["outer"], case["inner"])
    st["x"] = _normal(gen, shape, DTYPES[case["x"]])
    st["residual"] = _normal(gen, shape, DTYPES[case["x"]]) if case["residual"] else None
    st["seed"], st["offset"] = 0x9e3779b97f4a7c15 ^ int(seed), 5 * int(seed) + 1
    return st


# --------------------------------------------------------------------------
# plain forms: float32, elementary operations
# --------------------------------------------------------------------------
def _pieces(case, itemsize_rows):
    """(first query, queries, first key, keys, keys the first row sees) of parts of sequences small enough to hold."""
    out, a, c = [], 0, 0
    for lq, lk in zip(*_lengths(case)):
        step = max(1, CHUNK // max(1, itemsize_rows * lk))
        for r in range(0, lq, step):
            n = min(step, lq - r)
            out.append((a + r, n, c, lk, r + lk - lq + 1))
        a, c = a + lq, c + lk
    return out


def _by_head(x, g):
    """[rows, hkv * g, d] -> [hkv, rows * g, d]"""
    n, h, d = x.shape
    return x.float().view(n, h // g, g, d).permute(1, 0, 2, 3).reshape(h // g, n * g, d)


def _by_row(x, g):
    h, n, d = x.shape
    return x.view(h, n // g, g, d).permute(1, 0, 2, 3).reshape(n // g, h * g, d)


def _scores(st, qs, ks, c, lk, sees, g):
    """scale q k^T + bias with what a row does not see at -inf"""
    case = st["case"]
    x = torch.matmul(qs, ks.transpose(1, 2).contiguous()) * (1.0 / math.sqrt(case["dk"]))
    if st["bias"] is not None:
        x = x + st["bias"][c:c + lk]
    if case["causal"]:
        row = torch.arange(qs.shape[1], device="cuda") // g + sees
        x = x.masked_fill(torch.arange(lk, device="cuda") >= row[:, None], -math.inf)
    return x


def _attn_fwd_plain(st):
    case = st["case"]
    g, hkv, dt = case["hq"] // case["hkv"], case["hkv"], DTYPES[case["dtype"]]
    o = torch.empty((case["q"], case["hq"], case["dv"]), dtype=dt, device="cuda")
    lse = torch.empty((case["q"], case["hq"]), device="cuda")
    for a, n, c, lk, sees in _pieces(case, case["hq"]):
        qs = _by_head(st["q"][a:a + n], g)
        x = _scores(st, qs, _by_head(st["k"][c:c + lk], 1), c, lk, sees, g)
        m = x.amax(dim=2, keepdim=True)
        m = torch.where(m == -math.inf, 0.0, m)
        p = torch.exp(x - m)
        s = p.sum(dim=2, keepdim=True)
        y = torch.matmul(p, _by_head(st["v"][c:c + lk], 1)) / torch.where(s == 0.0, 1.0, s)
        o[a:a + n] = _by_row(y, g).to(dt)
        lse[a:a + n] = (m + torch.log(s)).view(hkv, n, g).permute(1, 0, 2).reshape(n, hkv * g)
    return o, lse


def _attn_bwd_plain(st):
    case = st["case"]
    g, hkv, dt = case["hq"] // case["hkv"], case["hkv"], DTYPES[case["dtype"]]
    scale = 1.0 / math.sqrt(case["dk"])
    gq = torch.empty((case["q"], case["hq"], case["dk"]), dtype=dt, device="cuda")
    gk = torch.zeros((case["k"], hkv, case["dk"]), device="cuda")
    gv = torch.zeros((case["k"], hkv, case["dv"]), device="cuda")
    for a, n, c, lk, sees in _pieces(case, case["hq"]):
        qs, ks = _by_head(st["q"][a:a + n], g), _by_head(st["k"][c:c + lk], 1)
        vs, gs = _by_head(st["v"][c:c + lk], 1), _by_head(st["go"][a:a + n], g)
        lse = st["lse"][a:a + n].view(n, hkv, g).permute(1, 0, 2).reshape(hkv, n * g, 1)
        delta = (gs * _by_head(st["o"][a:a + n], g)).sum(dim=2, keepdim=True)
        p = torch.exp(_scores(st, qs, ks, c, lk, sees, g) - torch.where(lse == -math.inf, 0.0, lse))
        ds = p * (torch.matmul(gs, vs.transpose(1, 2).contiguous()) - delta) * scale
        gq[a:a + n] = _by_row(torch.matmul(ds, ks), g).to(dt)
        gv[c:c + lk] += _by_row(torch.matmul(p.transpose(1, 2).contiguous(), gs), 1)
        gk[c:c + lk] += _by_row(torch.matmul(ds.transpose(1, 2).contiguous(), qs), 1)
    return gq, gk.to(dt), gv.to(dt)


def _turns(st):
    """cos and sin of every token and pair, from angles in float64"""
    pairs, axes = st["freq"].shape[0], st["case"]["axes"]
    pos = st["pos"].double().view(-1, axes)
    axis = torch.arange(pairs, device="cuda") * axes // max(1, pairs)
    angle = pos[:, axis] * st["freq"].double()
    return torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]


def _turn(x, cos, sin, interleaved):
    r = 2 * cos.shape[2]
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((y, x[..., r:]), dim=-1)


def _qk_plain(st):
    cos, sin = _turns(st)
    out = {}
    for n in "qk":
        x, w = st[n].float(), st[n + "w"]
        r = torch.rsqrt((x * x).mean(dim=2, keepdim=True) + QK_EPS)
        if st["case"]["op"] == "qk_fwd":
            out[n] = _turn(x * r * w, cos, sin, st["case"]["interleaved"]).to(st[n].dtype)
            continue
        gn = _turn(st["g" + n].float(), cos, -sin, st["case"]["interleaved"])
        out["gw" + n] = (gn * x * r).sum(dim=(0, 1))
        t = gn * w
        out["g" + n] = (r * (t - x * r * r * (t * x).mean(dim=2, keepdim=True))).to(st[n].dtype)
    return out


M32 = 0xffffffff


def _philox(blocks, offset, seed):
    """Four 32-bit words (in int64) of each counter (block, offset) under the key `seed`: Philox4x32, ten rounds."""
    c = [blocks & M32, blocks >> 32, torch.full_like(blocks, offset & M32), torch.full_like(blocks, (offset >> 32) & M32)]
    k0, k1 = seed & M32, (seed >> 32) & M32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57      # the low 64 bits, as two words
        c = [((b >> 32) & M32) ^ c[1] ^ k0, b & M32, ((a >> 32) & M32) ^ c[3] ^ k1, a & M32]
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    return c


def _threshold(p):
    return int(math.floor(p * 65536 + 0.5))


def _drop_plain(st):
    """Element e takes half-word e % 8 of block e // 8; it is kept where that is not below round(65536 p)."""
    case, x = st["case"], st["x"].view(-1)
    n, t = x.numel(), _threshold(case["p"])
    y = torch.empty(n, dtype=DTYPES[case["y"]], device="cuda")
    step = 1 << 25
    for a in range(0, n, step):
        e = min(n, a + step)
        words = _philox(torch.arange(a // 8, (e + 7) // 8, device="cuda"), st["offset"], st["seed"])
        halves = torch.stack([h for w in words for h in (w & 0xffff, w >> 16)], dim=1).view(-1)[:e - a]
        f = torch.where(halves >= t, x[a:e].float() * (65536.0 / (65536 - t)), 0.0)
        if st["residual"] is not None:
            f = f + st["residual"].view(-1)[a:e].float()
        y[a:e] = f.to(y.dtype)
    return y.view(st["x"].shape)


def run(state):
    case = state["case"]
    if not own:
        if case["op"] == "attn_fwd":
            o, lse = _attn_fwd_plain(state)
            return {"o": o, "lse": lse}
        if case["op"] == "attn_bwd":
            gq, gk, gv = _attn_bwd_plain(state)
            return {"gq": gq, "gk": gk, "gv": gv}
        return _qk_plain(state) if case["op"] in ("qk_fwd", "qk_bwd") else {"y": _drop_plain(state)}
    import spherical_disco_convolution_amd as sdc
    if case["op"] in ("attn_fwd", "attn_bwd"):
        q, k, v = state["q"], state["k"], state["v"]
        kw = dict(key_bias=state["bias"], causal=case["causal"])
        if case["mode"] == "packed":
            kw.update(cu_q=state["cu"], cu_k=state["cu"])
        else:       # a batch of equal lengths
            n = case["seqs"]
            q, k, v = (t.unflatten(0, (n, t.shape[0] // n)) for t in (q, k, v))
        if case["op"] == "attn_fwd":
            o, lse = sdc.attention_fwd(q, k, v, **kw)
            return {"o": o.view(state["q"].shape[:2] + o.shape[-1:]), "lse": lse.view(state["q"].shape[:2])}
        o, lse, go = (state[n].view(q.shape[:-2] + state[n].shape[1:]) for n in ("o", "lse", "go"))
        gq, gk, gv = sdc.attention_bwd(q, k, v, o, lse, go, **kw)
        return {"gq": gq.view(state["q"].shape), "gk": gk.view(state["k"].shape), "gv": gv.view(state["v"].shape)}
    if case["op"] in ("qk_fwd", "qk_bwd"):
        kw = dict(positions=state["pos"], inv_freq=state["freq"], interleaved=case["interleaved"], eps=QK_EPS)
        if case["op"] == "qk_fwd":
            q, k = sdc.qk_norm_rope_fwd(state["q"], state["k"], state["qw"], state["kw"], **kw)
            return {"q": q, "k": k}
        gq, gk, gwq, gwk = sdc.qk_norm_rope_bwd(state["q"], state["k"], state["gq"], state["gk"], state["qw"],
                                                state["kw"], **kw)
        return {"gwq": gwq, "gq": gq, "gwk": gwk, "gk": gk}
    if case["op"] == "drop_fwd":
        return {"y": sdc.dropout_fwd(state["x"], case["p"], state["seed"], offset=state["offset"],
                                     residual=state["residual"], out_dtype=DTYPES[case["y"]])}
    return {"y": sdc.dropout_bwd(state["x"], case["p"], state["seed"], offset=state["offset"],
                                 gx_dtype=DTYPES[case["y"]])}


def work(case):
    size = {F32: 4, BF16: 2}
    if case["op"] in ("attn_fwd", "attn_bwd"):
        s = size[case["dtype"]]
        dk, dv, hq, hkv, tq, tk = (case[n] for n in ("dk", "dv", "hq", "hkv", "q", "k"))
        pairs = 0
        for lq, lk in zip(*_lengths(case)):
            full = lq * lk
            if case["causal"]:     # row i of lq sees i + 1 + lk - lq keys
                full = lq * (lk - lq) + lq * (lq + 1) // 2
            pairs += full
        nbytes = s * (tq * hq * (dk + dv) + tk * hkv * (dk + dv)) + 4 * tq * hq + (4 * tk if case["bias"] else 0)
        if case["op"] == "attn_fwd":
            return {"bytes": nbytes, "flops": 2 * pairs * hq * (dk + dv)}
        nbytes += s * (tq * hq * (dk + dv) + tk * hkv * (dk + dv))
        return {"bytes": nbytes, "flops": 2 * pairs * hq * (3 * dk + 2 * dv)}
    if case["op"] in ("qk_fwd", "qk_bwd"):
        e = case["tokens"] * (case["hq"] + case["hkv"]) * case["d"]
        other = 4 * (case["tokens"] * case["axes"] + case["rot"] // 2) + 8 * case["d"]
        if case["op"] == "qk_fwd":
            return {"bytes": 2 * e * size[case["dtype"]] + other, "flops": 7 * e}
        return {"bytes": 3 * e * size[case["dtype"]] + other + 8 * case["d"], "flops": 14 * e}
    e = case["outer"] * case["inner"]
    sx, sy = size[case["x"]], size[case["y"]]
    return {"bytes": e * (sx + sy + (sx if case["residual"] else 0)), "flops": 2 * e}


# --------------------------------------------------------------------------
# the definitions in float64
# --------------------------------------------------------------------------
def _attn_exact(st):
    """One head at a time, softmax from the scores' own logarithm of the sum."""
    case = st["case"]
    tq, tk, hq, hkv = case["q"], case["k"], case["hq"], case["hkv"]
    scale = case["dk"] ** -0.5
    bwd = case["op"] == "attn_bwd"
    new = dict(dtype=torch.float64, device="cuda")
    o, lse = torch.zeros((tq, hq, case["dv"]), **new), torch.zeros((tq, hq), **new)
    gq, gk, gv = (torch.zeros((n, h, d), **new) for n, h, d in
                  ((tq, hq, case["dk"]), (tk, hkv, case["dk"]), (tk, hkv, case["dv"])))
    a = c = 0
    for lq, lk in zip(*_lengths(case)):
        key = torch.arange(lk, device="cuda")
        for h in range(hq):
            kv = h * hkv // hq
            ks, vs = st["k"][c:c + lk, kv].double(), st["v"][c:c + lk, kv].double()
            kt, vt = ks.t().contiguous(), vs.t().contiguous()
            for r in range(0, lq, 4096):
                rows = slice(a + r, a + min(lq, r + 4096))
                qs = st["q"][rows, h].double()
                x = qs @ kt * scale
                if case["bias"]:
                    x += st["bias"][None, c:c + lk].double()
                if case["causal"]:
                    last = torch.arange(rows.start - a, rows.stop - a, device="cuda") + (lk - lq)
                    x[key[None, :] > last[:, None]] = -math.inf
                if not bwd:
                    l = torch.logsumexp(x, dim=1)
                    lse[rows, h] = l
                    o[rows, h] = torch.exp(x - torch.nan_to_num(l, neginf=0.0)[:, None]) @ vs
                    continue
                p = torch.exp(x - torch.nan_to_num(st["lse"][rows, h].double(), neginf=0.0)[:, None])
                g = st["go"][rows, h].double()
                ds = p * (g @ vt - (g * st["o"][rows, h].double()).sum(1)[:, None])
                gq[rows, h] = ds @ ks * scale
                gk[c:c + lk, kv] += ds.t().contiguous() @ qs * scale
                gv[c:c + lk, kv] += p.t().contiguous() @ g
        a, c = a + lq, c + lk
    return {"gq": gq, "gk": gk, "gv": gv} if bwd else {"o": o, "lse": lse}


def _qk_exact(st):
    """Pairs as complex numbers, turned by a product."""
    case = st["case"]
    d, rot, axes = case["d"], case["rot"], case["axes"]
    half = rot // 2
    angle = torch.stack([st["pos"].double().view(-1, axes)[:, p * axes // half] * float(st["freq"][p])
                         for p in range(half)], dim=1) if half else torch.zeros((case["tokens"], 0), device="cuda")
    unit = torch.polar(torch.ones_like(angle, dtype=torch.float64), angle.double())[:, None]
    first = torch.arange(half, device="cuda") * 2 if case["interleaved"] else torch.arange(half, device="cuda")
    second = first + (1 if case["interleaved"] else half)
    out = {}
    for n in ("q", "k"):
        x, w = st[n].double(), st[n + "w"].double()
        y = (st["g" + n].double() if case["op"] == "qk_bwd" else
             w * x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / d + QK_EPS)).clone()
        z = torch.complex(y[..., first], y[..., second]) * (unit.conj() if case["op"] == "qk_bwd" else unit)
        y[..., first], y[..., second] = z.real, z.imag
        if case["op"] == "qk_fwd":
            out[n] = y
            continue
        rms = torch.sqrt(x.pow(2).sum(-1, keepdim=True) / d + QK_EPS)
        h = x / rms
        out["gw" + n] = torch.einsum("thd,thd->d", y, h)
        y = y * w
        out["g" + n] = (y - h * (y * h).sum(-1, keepdim=True) / d) / rms
    return out


def _drop_exact(st):
    """The generator in 16-bit limbs: a product of words is summed from four products of halves."""
    case = st["case"]
    n, t = st["x"].numel(), _threshold(case["p"])
    half = torch.empty(n + 7 & ~7, dtype=torch.int32, device="cuda")

    def product(m, v):
        lo, hi = (m & 0xffff) * v, (m >> 16) * v         # 48 bits each
        mid = hi + (lo >> 16)
        return (mid >> 16) & M32, ((mid & 0xffff) << 16) | (lo & 0xffff)

    for a in range(0, half.numel() // 8, 1 << 22):
        block = torch.arange(a, min(half.numel() // 8, a + (1 << 22)), device="cuda")
        w, x, y, z = block % (1 << 32), block // (1 << 32), block * 0 + st["offset"] % (1 << 32), \
            block * 0 + (st["offset"] >> 32) % (1 << 32)
        for r in range(10):
            k0 = ((st["seed"] % (1 << 32)) + r * 0x9E3779B9) % (1 << 32)
            k1 = ((st["seed"] >> 32) % (1 << 32) + r * 0xBB67AE85) % (1 << 32)
            (h0, l0), (h1, l1) = product(0xD2511F53, w), product(0xCD9E8D57, y)
            w, x, y, z = h1 ^ x ^ k0, l1, h0 ^ z ^ k1, l0
        part = half[8 * a:8 * (a + block.numel())].view(-1, 8)
        for i, word in enumerate((w, x, y, z)):
            part[:, 2 * i], part[:, 2 * i + 1] = (word % 65536).int(), (word // 65536).int()
    y = st["x"].double().flatten()
    y = y * (half[:n] >= t) / (1.0 - t / 65536.0)
    if st["residual"] is not None:
        y += st["residual"].flatten().double()
    return {"y": y.view(st["x"].shape)}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("attn_fwd", "attn_bwd"):
        return _attn_exact(st)
    return _qk_exact(st) if case["op"] in ("qk_fwd", "qk_bwd") else _drop_exact(st)
