"""Cases for the operators that train and run the cross-attention of the sparse tokens: the attention
itself over packed groups (forward and backward), the per-head norm of its queries and keys with the
rotary positions of the tokens' (t, y, x) coordinates in the same pass (forward and backward), and the
global norm and clipping of the gradients of the whole adapter stack.

`run` computes a case in plain torch operations (own = False) or through the framework (own = True).
"""
import math

import torch

own = False

# ---------------------------------------------------------------- cases
# Group lengths: group 0 has the full length, the others a fixed share of it, so a batch is ragged.
_SHARES = (1.0, 0.43, 0.0, 0.87, 0.61, 0.99, 0.12, 0.75)


def _lens(G, longest, shift):
    return [longest if g == 0 else int(longest * _SHARES[(g * (3 + shift)) % 8]) for g in range(G)]


def _offsets(lens):
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    return off


def listed():
    return [
        # a handful of landmark queries per video over a short clip's tokens: all latency
        {"name": "attn fwd tiny", "op": "attn_fwd", "G": 2, "max_q": 3, "max_kv": 77, "Hq": 2, "Hkv": 2, "d": 32, "keep": 1.0},
        # one CLS token over every token of a whole long video, 256 channels in 4 heads
        {"name": "attn fwd cls long video", "op": "attn_fwd", "G": 1, "max_q": 1, "max_kv": 282624, "Hq": 4, "Hkv": 4, "d": 64, "keep": 1.0},
        # every kept token of eight videos asks a few dozen encoder states of its video
        {"name": "attn fwd tokens to states", "op": "attn_fwd", "G": 8, "max_q": 6144, "max_kv": 77, "Hq": 4, "Hkv": 4, "d": 64, "keep": 1.0},
        # long queries over long states, shared key heads, some of the states dropped
        {"name": "attn fwd long", "op": "attn_fwd", "G": 2, "max_q": 4096, "max_kv": 8192, "Hq": 8, "Hkv": 2, "d": 128, "keep": 0.9},
        # training: aux tokens over clips
        {"name": "attn bwd aux", "op": "attn_bwd", "G": 4, "max_q": 16, "max_kv": 9000, "Hq": 4, "Hkv": 4, "d": 64, "keep": 1.0},
        # training: tokens to tokens of another stream, ragged
        {"name": "attn bwd clips", "op": "attn_bwd", "G": 8, "max_q": 1001, "max_kv": 1543, "Hq": 4, "Hkv": 4, "d": 64, "keep": 0.9},
        # training: the largest
        {"name": "attn bwd long", "op": "attn_bwd", "G": 2, "max_q": 2048, "max_kv": 4096, "Hq": 8, "Hkv": 2, "d": 128, "keep": 1.0},
        # norm and rotation of a few tokens (serving)
        {"name": "qk fwd few", "op": "qk_fwd", "nq": 4, "nk": 231, "Hq": 4, "Hkv": 4, "d": 64, "rot": 64, "layout": "half", "axes": 1, "dtype": "bf16"},
        # of a batch of frames against a long video, three axes, part of the head
        {"name": "qk fwd video", "op": "qk_fwd", "nq": 49152, "nk": 282624, "Hq": 4, "Hkv": 4, "d": 64, "rot": 48, "layout": "half", "axes": 3, "dtype": "bf16"},
        # its gradients
        {"name": "qk bwd batch", "op": "qk_bwd", "nq": 49152, "nk": 98317, "Hq": 8, "Hkv": 2, "d": 128, "rot": 96, "layout": "interleaved", "axes": 3, "dtype": "bf16"},
        # gradients of one small convolution
        {"name": "clip one layer", "op": "clip", "layers": 1, "D": 128, "R": 64, "bf16": 0, "over": 4.0},
        # gradients of the adapters of a 24-block backbone
        {"name": "clip adapters", "op": "clip", "layers": 24, "D": 1024, "R": 256, "bf16": 0, "over": 4.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_bwd", "qk_fwd", "qk_bwd", "clip", "attn_fwd", "attn_bwd"])
    if op in ("attn_fwd", "attn_bwd"):
        big = op == "attn_fwd"
        while True:
            r = rng.choice([1, 1, 2, 3, 4])
            Hkv = rng.choice([1, 2, 4])
            c = {"op": op, "G": rng.choice([1, 1, 2, 3, 5, 8]), "max_q": _log(rng, 1, 6000), "max_kv": _log(rng, 1, 250000 if big else 20000),
                 "Hq": Hkv * r, "Hkv": Hkv, "d": rng.choice([16, 32, 40, 64, 64, 80, 96, 128, 128]), "keep": rng.choice([1.0, 1.0, 0.9, 0.5])}
            if c["G"] * c["Hq"] * c["max_q"] * c["max_kv"] <= (5e8 if big else 1.2e8) and c["G"] * c["Hkv"] * c["d"] * c["max_kv"] <= 7.2e7:
                return c
    if op in ("qk_fwd", "qk_bwd"):
        while True:
            d = rng.choice([16, 32, 64, 64, 80, 128, 128, 256])
            Hkv = rng.choice([1, 2, 4])
            c = {"op": op, "nq": _log(rng, 1, 60000), "nk": _log(rng, 1, 280000), "Hq": Hkv * rng.choice([1, 2, 4]), "Hkv": Hkv, "d": d,
                 "rot": 16 * rng.randint(1, d // 16), "layout": rng.choice(["half", "interleaved"]), "axes": rng.choice([1, 2, 3]),
                 "dtype": rng.choice(["bf16", "bf16", "f32"])}
            if (c["nq"] * c["Hq"] + c["nk"] * c["Hkv"]) * d * (1 if c["dtype"] == "bf16" else 2) <= 7.0e7:
                return c
    return {"op": "clip", "layers": rng.randint(1, 24), "D": rng.choice([64, 100, 384, 768, 1024]), "R": rng.choice([16, 33, 64, 128, 256]),
            "bf16": rng.choice([0, 1]), "over": rng.choice([0.5, 4.0])}


# ---------------------------------------------------------------- inputs
def _normal(gen, shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _sizes(case):
    ql, kl = _lens(case["G"], case["max_q"], 0), _lens(case["G"], case["max_kv"], 2)
    return _offsets(ql), _offsets(kl)


def _adapter_shapes(case):
    D, R = case["D"], case["R"]
    return [s for _ in range(case["layers"]) for s in ((R, D), (R, 9, R), (R,), (D, R))]


def _frequencies(case):
    """Base 10,000, each axis with its own run from fast to slow; scaled by 1/4 for positions four times as far."""
    pairs, axes = case["rot"] // 2, case["axes"]
    split = [pairs // axes + (1 if a < pairs % axes else 0) for a in range(axes)]
    freq = [10000.0 ** (-i / n) / 4 for n in split for i in range(n)]
    return split, torch.tensor(freq, dtype=torch.float64, device="cuda")


def _positions(gen, n, axes):
    """Token coordinates (t, y, x); a single axis counts the tokens of a long stream."""
    if axes == 1:
        return torch.arange(n, dtype=torch.int32, device="cuda").reshape(n, 1)
    hi = (4096, 16, 16) if axes == 3 else (64, 64)
    return torch.stack([torch.randint(0, h, (n,), generator=gen, device="cuda", dtype=torch.int32) for h in hi], 1).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    if op in ("attn_fwd", "attn_bwd"):
        qo, ko = _sizes(case)
        Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
        s["q_off"] = torch.tensor(qo, dtype=torch.int32, device="cuda")
        s["kv_off"] = torch.tensor(ko, dtype=torch.int32, device="cuda")
        s["Q"] = _normal(gen, (qo[-1], Hq, d), scale=1.5)
        s["K"] = _normal(gen, (ko[-1], Hkv, d))
        s["V"] = _normal(gen, (ko[-1], Hkv, d))
        s["keep"] = None
        if case["keep"] < 1:
            s["keep"] = (torch.rand((ko[-1],), generator=gen, device="cuda") < case["keep"]).to(torch.uint8)
        if op == "attn_bwd":  # what the forward pass left behind
            s["dO"] = _normal(gen, (qo[-1], Hq, d))
            O, L = _attn_plain(s["Q"], s["K"], s["V"], s["q_off"], s["kv_off"], case, s["keep"])
            s["O"], s["L"] = O, L
    elif op in ("qk_fwd", "qk_bwd"):
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        d = case["d"]
        s["Q"] = _normal(gen, (case["nq"], case["Hq"], d), dt, 2.0)
        s["K"] = _normal(gen, (case["nk"], case["Hkv"], d), dt, 0.5)
        s["wq"] = 1.0 + 0.2 * torch.randn((d,), generator=gen, device="cuda")
        s["wk"] = 1.0 + 0.2 * torch.randn((d,), generator=gen, device="cuda")
        s["pq"], s["pk"] = _positions(gen, case["nq"], case["axes"]), _positions(gen, case["nk"], case["axes"])
        s["split"], s["freq"] = _frequencies(case)
        if op == "qk_bwd":
            s["dYq"] = _normal(gen, (case["nq"], case["Hq"], d), dt)
            s["dYk"] = _normal(gen, (case["nk"], case["Hkv"], d), dt)
    else:
        shapes = _adapter_shapes(case)
        sizes = [math.prod(x) for x in shapes]
        # the gradients of the up- and down-projections in bf16 where the case says so, the rest in fp32
        kind = [case["bf16"] and len(x) == 2 for x in shapes]
        total = {b: sum(n for n, k in zip(sizes, kind) if bool(k) == b) for b in (False, True)}
        flat = {b: _normal(gen, (total[b],), torch.bfloat16 if b else torch.float32, 0.01) for b in (False, True)}
        out = {b: torch.empty_like(flat[b]) for b in flat}
        s["grads"], s["outs"], at = [], [], {False: 0, True: 0}
        for shape, n, k in zip(shapes, sizes, kind):
            b = bool(k)
            s["grads"].append(flat[b][at[b]:at[b] + n].view(shape))
            s["outs"].append(out[b][at[b]:at[b] + n].view(shape))
            at[b] += n
        s["out"] = [o for o in out.values() if o.numel()]
        s["max_norm"] = 0.01 * math.sqrt(sum(sizes)) / case["over"]
    return s


# ---------------------------------------------------------------- plain forms
def _padded(off, longest, n):
    """Row of each (group, position), which of them exist, and (group, position) of each row."""
    o = off.long()
    at = torch.arange(longest, device=off.device)
    there = at[None, :] < (o[1:] - o[:-1])[:, None]
    rows = (o[:-1, None] + at[None, :]).clamp(max=max(n - 1, 0))
    row = torch.arange(n, device=off.device)
    group = torch.bucketize(row, o[1:], right=True)
    return rows, there, group, row - o[group]


def _attn_parts(Q, K, q_off, kv_off, case, keep):
    """Row and column tables and the scores [G, Hkv, r, Lq, Lk] in fp32 with the absent keys at -inf."""
    G, Hq, Hkv, d = case["G"], case["Hq"], case["Hkv"], case["d"]
    qr, _, qg, qp = _padded(q_off, case["max_q"], Q.shape[0])
    kr, kt, kg, kp = _padded(kv_off, case["max_kv"], K.shape[0])
    if keep is not None:
        kt = kt & (keep[kr] != 0)
    q = Q[qr].float().view(G, case["max_q"], Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4)
    k = K[kr].float().permute(0, 2, 3, 1)[:, :, None]
    s = torch.matmul(q, k) * (1.0 / math.sqrt(d))
    s = s.masked_fill_(~kt[:, None, None, None, :], -math.inf)
    return s, (qr, qg, qp), (kr, kg, kp)


def _softmax(s):
    """(weights, log of the sum) of each row in place of the scores; a row without keys has weights 0."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    p = p.mul_(torch.where(z > 0, 1.0 / z, torch.zeros_like(z)))
    return p, (m + z.log())[..., 0]


def _rows(x, table):
    """[G, H.., L, d] back to packed rows [n, H, d]."""
    _, g, at = table
    x = x.flatten(1, -3) if x.dim() > 4 else x
    return x.transpose(1, 2)[g, at]


def _attn_plain(Q, K, V, q_off, kv_off, case, keep):
    s, qt, kt = _attn_parts(Q, K, q_off, kv_off, case, keep)
    p, L = _softmax(s)
    o = torch.matmul(p, V[kt[0]].float().permute(0, 2, 1, 3)[:, :, None])
    L = L.flatten(1, 2).transpose(1, 2)[qt[1], qt[2]]
    return _rows(o, qt).to(Q.dtype).contiguous(), L.contiguous()


def _attn_plain_bwd(s):
    case = s["case"]
    Q, K, V, dO = s["Q"], s["K"], s["V"], s["dO"]
    G, Hq, Hkv, d = case["G"], case["Hq"], case["Hkv"], case["d"]
    sc, qt, kt = _attn_parts(Q, K, s["q_off"], s["kv_off"], case, s["keep"])
    p, _ = _softmax(sc)
    qn = (s["q_off"][1:] - s["q_off"][:-1]).long()
    there = (torch.arange(case["max_q"], device=Q.device)[None, :] < qn[:, None]).float()
    go = (dO[qt[0]].float() * there[:, :, None, None]).view(G, case["max_q"], Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4)
    v = V[kt[0]].float().permute(0, 2, 3, 1)[:, :, None]
    dv = torch.matmul(p.transpose(-1, -2), go).sum(2)
    dp = torch.matmul(go, v)
    ds = dp.sub_((p * dp).sum(-1, keepdim=True)).mul_(p).mul_(1.0 / math.sqrt(d))
    q = Q[qt[0]].float().view(G, case["max_q"], Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2)
    dq = torch.matmul(ds, K[kt[0]].float().permute(0, 2, 1, 3)[:, :, None])
    return [_rows(dq, qt).to(Q.dtype), _rows(dk, kt).to(K.dtype), _rows(dv, kt).to(V.dtype)]


def _turns(pos, split, freq):
    """cos and sin [n, 1, pairs] of position x frequency; the angle in 64 bits."""
    axis = torch.repeat_interleave(torch.arange(len(split), device=pos.device), torch.tensor(split, device=pos.device))
    a = pos.double()[:, axis] * freq
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _pairs(x, rot, layout):
    h = x[..., :rot]
    return (h[..., :rot // 2], h[..., rot // 2:]) if layout == "half" else (h[..., 0::2], h[..., 1::2])


def _joined(a, b, rest, layout):
    h = torch.cat([a, b], -1) if layout == "half" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([h, rest], -1)


_EPS = 1e-6


def _qk_plain(x, pos, w, s):
    case = s["case"]
    f = x.float()
    y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + _EPS) * w
    c, n = _turns(pos, s["split"], s["freq"])
    a, b = _pairs(y, case["rot"], case["layout"])
    return _joined(a * c - b * n, a * n + b * c, y[..., case["rot"]:], case["layout"]).to(x.dtype)


def _qk_plain_bwd(dy, x, pos, w, s):
    case = s["case"]
    f, g = x.float(), dy.float()
    c, n = _turns(pos, s["split"], s["freq"])
    a, b = _pairs(g, case["rot"], case["layout"])
    g = _joined(a * c + b * n, b * c - a * n, g[..., case["rot"]:], case["layout"])
    r = torch.rsqrt(f.square().mean(-1, keepdim=True) + _EPS)
    xh = f * r
    dw = (g * xh).sum((0, 1), dtype=torch.float64).float()
    gw = g * w
    return (r * (gw - xh * (gw * xh).mean(-1, keepdim=True))).to(x.dtype), dw


def _clip_plain(s):
    norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum().sqrt().float()
    scale = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    torch._foreach_copy_(s["outs"], [(g.float() * scale).to(g.dtype) for g in s["grads"]])
    return [norm] + s["out"]


# ---------------------------------------------------------------- one pass
def run(s):
    op, case = s["op"], s["case"]
    if not own:
        if op == "attn_fwd":
            return list(_attn_plain(s["Q"], s["K"], s["V"], s["q_off"], s["kv_off"], case, s["keep"]))
        if op == "attn_bwd":
            return _attn_plain_bwd(s)
        if op == "qk_fwd":
            return [_qk_plain(s["Q"], s["pq"], s["wq"], s), _qk_plain(s["K"], s["pk"], s["wk"], s)]
        if op == "qk_bwd":
            dQ, dwq = _qk_plain_bwd(s["dYq"], s["Q"], s["pq"], s["wq"], s)
            dK, dwk = _qk_plain_bwd(s["dYk"], s["K"], s["pk"], s["wk"], s)
            return [dQ, dK, dwq, dwk]
        return _clip_plain(s)
    from sparse_convolution_pruned_b200 import svconv as sv
    if op == "attn_fwd":
        return list(sv.svconv_cross_attn_fwd(s["Q"], s["K"], s["V"], s["q_off"], s["kv_off"], max_q=case["max_q"], max_kv=case["max_kv"], kv_keep=s["keep"]))
    if op == "attn_bwd":
        return list(sv.svconv_cross_attn_bwd(s["dO"], s["Q"], s["K"], s["V"], s["O"], s["L"], s["q_off"], s["kv_off"],
                                             max_q=case["max_q"], max_kv=case["max_kv"], kv_keep=s["keep"]))
    if op == "qk_fwd":
        return list(sv.svconv_qk_norm_rope_fwd(s["Q"], s["K"], s["pq"], s["pk"], s["freq"], wq=s["wq"], wk=s["wk"], eps=_EPS,
                                               layout=case["layout"], axis_pairs=s["split"]))
    if op == "qk_bwd":
        return list(sv.svconv_qk_norm_rope_bwd(s["dYq"], s["dYk"], s["Q"], s["K"], s["pq"], s["pk"], s["freq"], wq=s["wq"], wk=s["wk"],
                                               eps=_EPS, layout=case["layout"], axis_pairs=s["split"]))
    return [sv.svconv_clip_grads(s["grads"], s["max_norm"], out=s["outs"])] + s["out"]


# ---------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op in ("attn_fwd", "attn_bwd"):
        ql, kl = _lens(case["G"], case["max_q"], 0), _lens(case["G"], case["max_kv"], 2)
        pairs = sum(a * b for a, b in zip(ql, kl)) * case["Hq"]
        nq, nk, d = sum(ql) * case["Hq"], sum(kl) * case["Hkv"], case["d"]
        keep = sum(kl) if case["keep"] < 1 else 0
        if op == "attn_fwd":
            return {"bytes": 2 * d * (2 * nq + 2 * nk) + 4 * nq + keep, "flops": 4 * pairs * d}
        return {"bytes": 2 * d * (4 * nq + 4 * nk) + 4 * nq + keep, "flops": 10 * pairs * d}
    if op in ("qk_fwd", "qk_bwd"):
        values = (case["nq"] * case["Hq"] + case["nk"] * case["Hkv"]) * case["d"]
        each = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": values * each * (2 if op == "qk_fwd" else 3) + 4 * case["axes"] * (case["nq"] + case["nk"]),
                "flops": values * (8 if op == "qk_fwd" else 16)}
    sizes = [(math.prod(x), 2 if case["bf16"] and len(x) == 2 else 4) for x in _adapter_shapes(case)]
    return {"bytes": sum(2 * n * b for n, b in sizes), "flops": sum(3 * n for n, _ in sizes)}


# ---------------------------------------------------------------- from the definitions, in 64 bits
def _exact_attn(s, case):
    qo, ko = _sizes(case)
    Q, K, V = (s[k].double() for k in ("Q", "K", "V"))
    nq, Hq, d = Q.shape
    r = Hq // case["Hkv"]
    O, L = torch.zeros_like(Q), torch.full((nq, Hq), -math.inf, dtype=torch.float64, device="cuda")
    grads = [torch.zeros_like(t) for t in (Q, K, V)]
    for g in range(case["G"]):
        a, b = slice(qo[g], qo[g + 1]), torch.arange(ko[g], ko[g + 1], device="cuda")
        if s["keep"] is not None:
            b = b[s["keep"][b] != 0]
        if b.numel() == 0 or qo[g] == qo[g + 1]:
            continue
        for h in range(Hq):
            q, k, v = Q[a, h], K[b, h // r], V[b, h // r]
            z = q @ k.T / math.sqrt(d)
            L[a, h] = torch.logsumexp(z, 1)
            P = torch.exp(z - L[a, h][:, None])
            O[a, h] = P @ v
            if case["op"] == "attn_bwd":
                do = s["dO"][a, h].double()
                dS = P * (do @ v.T - (do * O[a, h]).sum(1, keepdim=True)) / math.sqrt(d)
                grads[0][a, h] = dS @ k
                grads[1][b, h // r] += dS.T @ q
                grads[2][b, h // r] += P.T @ do
    return [O, L] if case["op"] == "attn_fwd" else grads


def _exact_qk(x, dy, pos, w, s, case):
    """The norm and the rotation as a matrix on each pair, and their transposes."""
    x, w = x.double(), w.double()
    n, H, d = x.shape
    rot = case["rot"]
    at = torch.arange(rot // 2, device="cuda")
    first, second = (at, at + rot // 2) if case["layout"] == "half" else (2 * at, 2 * at + 1)
    axis = torch.tensor([a for a, m in enumerate(s["split"]) for _ in range(m)], device="cuda")
    ang = (pos.double()[:, axis] * s["freq"][None])[:, None, :]
    co, si = torch.cos(ang), torch.sin(ang)
    norm = torch.sqrt((x * x).sum(-1, keepdim=True) / d + _EPS)
    unit = x / norm
    if dy is None:
        y = unit * w
        out = y.clone()
        out[..., first] = y[..., first] * co - y[..., second] * si
        out[..., second] = y[..., second] * co + y[..., first] * si
        return out, None
    g0 = dy.double()
    g = g0.clone()
    g[..., first] = g0[..., first] * co + g0[..., second] * si
    g[..., second] = g0[..., second] * co - g0[..., first] * si
    dw = (g * unit).reshape(-1, d).sum(0)
    g = g * w
    return (g - unit * ((g * unit).sum(-1, keepdim=True) / d)) / norm, dw


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("attn_fwd", "attn_bwd"):
        return _exact_attn(s, case)
    if op == "qk_fwd":
        return [_exact_qk(s["Q"], None, s["pq"], s["wq"], s, case)[0], _exact_qk(s["K"], None, s["pk"], s["wk"], s, case)[0]]
    if op == "qk_bwd":
        dQ, dwq = _exact_qk(s["Q"], s["dYq"], s["pq"], s["wq"], s, case)
        dK, dwk = _exact_qk(s["K"], s["dYk"], s["pk"], s["wk"], s, case)
        return [dQ, dK, dwq, dwk]
    norm = math.sqrt(sum(float((g.double() ** 2).sum()) for g in s["grads"]))
    scale = min(1.0, s["max_norm"] / (norm + 1e-6))
    flat = {}
    for g in s["grads"]:
        flat.setdefault(g.dtype, []).append(g.double().flatten() * scale)
    order = [t for t in (torch.float32, torch.bfloat16) if t in flat]
    return [torch.tensor(norm, dtype=torch.float64)] + [torch.cat(flat[t]) for t in order]
