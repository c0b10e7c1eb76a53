"""svconv_qk_norm_rope_fwd / _bwd against the formulas in 64 bits.

Bounds: everything is fp32 and rounds once at the end, so an output is off by at most half a step of
its type (u) of its value, plus fp32 terms: ~16 operations of 2^-24 each on values no larger than
|u_a| + |u_b| (forward) or rstd (|g w| + |xhat| |dot|) (backward), and 2^-22 for a sine or cosine.
dw sums n H products, each off by a few 2^-24 of its magnitude, in fp32 chains of at most a few
hundred additions.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
E32 = 2.0 ** -20


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_convolution_pruned_b200 import build, svconv
    build.build()
    return svconv


def half_step(dt):
    return torch.finfo(dt).eps / 2


def make(seed, n, H, d, dt, axes, far=False, strided=False):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
    x = (2 * rnd(n, H + (1 if strided else 0), d)).to(dt)[:, :H]
    pos = torch.randint(0, 2 ** 30 if far else 5000, (n, axes), generator=gen, device="cuda", dtype=torch.int32)
    if n > 2:
        pos[1] = -pos[1]
    return {"x": x, "pos": pos, "w": 1 + 0.3 * rnd(d), "dy": rnd(n, H, d).to(dt)}


def reference(s, split, freq, layout, eps, use_w=True):
    x, dy = s["x"].double(), s["dy"].double()
    w = s["w"].double() if use_w else torch.ones_like(s["w"]).double()
    n, H, d = x.shape
    pairs = len(freq)
    at = torch.arange(pairs, device="cuda")
    a, b = (at, at + pairs) if layout == "half" else (2 * at, 2 * at + 1)
    axis = torch.tensor([i for i, m in enumerate(split) for _ in range(m)], dtype=torch.long, device="cuda")
    ang = (s["pos"].double()[:, axis] * freq)[:, None]
    c, z = ang.cos(), ang.sin()
    rstd = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    xh = x * rstd
    u = xh * w
    y, ty = u.clone(), u.abs()
    y[..., a], y[..., b] = u[..., a] * c - u[..., b] * z, u[..., a] * z + u[..., b] * c
    m = u[..., a].abs() + u[..., b].abs()
    ty[..., a], ty[..., b] = m, m
    g, tg = dy.clone(), dy.abs()
    g[..., a], g[..., b] = dy[..., a] * c + dy[..., b] * z, dy[..., b] * c - dy[..., a] * z
    m = dy[..., a].abs() + dy[..., b].abs()
    tg[..., a], tg[..., b] = m, m
    gw = g * w
    dot = (gw * xh).mean(-1, keepdim=True)
    dx = rstd * (gw - xh * dot)
    tdx = rstd * (tg * w.abs() + xh.abs() * (tg * w.abs() * xh.abs()).mean(-1, keepdim=True))
    return {"y": y, "dx": dx, "dw": (g * xh).sum((0, 1))}, {"y": ty, "dx": tdx, "dw": (tg * xh.abs()).sum((0, 1))}


def close(got, ref, mag, dt, what):
    over = (got.double() - ref).abs() - half_step(dt) * ref.abs() * (1 + 2 ** -6) - E32 * mag - 1e-30
    assert over.numel() == 0 or float(over.max()) <= 0, f"{what}: {float(over.max()):.3e} over its bound"


CASES = [
    # nq, nk, Hq, Hkv, d, rot, layout, split, dtype, strided
    (1, 1, 1, 1, 8, 0, "half", [0], "bf16", False),
    (1, 5, 1, 1, 16, 16, "interleaved", [8], "bf16", False),
    (7, 33, 4, 4, 64, 64, "half", [32], "bf16", False),
    (100, 1001, 4, 2, 64, 48, "half", [8, 8, 8], "bf16", True),
    (1001, 100, 8, 2, 128, 96, "interleaved", [20, 0, 28], "bf16", True),
    (65, 257, 16, 1, 128, 128, "half", [64], "f32", False),
    (65, 257, 3, 3, 80, 32, "half", [7, 9], "f32", True),
    (65, 257, 5, 5, 24, 16, "interleaved", [8], "bf16", False),
    (31, 300, 2, 1, 256, 256, "half", [128], "bf16", False),
    (31, 300, 9, 3, 256, 240, "interleaved", [40, 40, 40], "f32", False),
    (0, 300, 2, 2, 64, 64, "half", [32], "bf16", False),
    (50, 0, 2, 2, 64, 64, "half", [32], "f32", False),
    (20000, 50001, 2, 1, 64, 32, "half", [6, 5, 5], "bf16", False),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_against_the_formulas(sv, i):
    nq, nk, Hq, Hkv, d, rot, layout, split, dtype, strided = CASES[i]
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    axes = len(split)
    q, k = make(i, nq, Hq, d, dt, axes, strided=strided), make(50 + i, nk, Hkv, d, dt, axes, strided=strided)
    freq = (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(rot // 2, 1))).cuda()
    kw = dict(wq=q["w"], wk=k["w"], eps=1e-5, layout=layout, axis_pairs=split)
    y = sv.svconv_qk_norm_rope_fwd(q["x"], k["x"], q["pos"], k["pos"], freq, **kw)
    g = sv.svconv_qk_norm_rope_bwd(q["dy"], k["dy"], q["x"], k["x"], q["pos"], k["pos"], freq, **kw)
    g2 = sv.svconv_qk_norm_rope_bwd(q["dy"], k["dy"], q["x"], k["x"], q["pos"], k["pos"], freq, **kw)
    torch.cuda.synchronize()
    for a, b in zip(g, g2):
        assert torch.equal(a, b)
    for j, s in enumerate((q, k)):
        ref, mag = reference(s, split, freq, layout, 1e-5)
        close(y[j], ref["y"], mag["y"], dt, f"{CASES[i]} y{j}")
        close(g[j], ref["dx"], mag["dx"], dt, f"{CASES[i]} dx{j}")
        close(g[2 + j], ref["dw"], mag["dw"], torch.float32, f"{CASES[i]} dw{j}")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_positions_and_no_weight(sv, layout):
    """Positions up to 2^30: the angle is formed in 64 bits."""
    q, k = make(1, 200, 2, 64, torch.float32, 1, far=True), make(2, 300, 2, 64, torch.float32, 1, far=True)
    freq = (500000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).cuda()
    y = sv.svconv_qk_norm_rope_fwd(q["x"], k["x"], q["pos"], k["pos"], freq, layout=layout)
    g = sv.svconv_qk_norm_rope_bwd(q["dy"], k["dy"], q["x"], k["x"], q["pos"], k["pos"], freq, layout=layout, want_dw=False)
    assert g[2] is None and g[3] is None
    for j, s in enumerate((q, k)):
        ref, mag = reference(s, [32], freq, layout, 1e-6, use_w=False)
        close(y[j], ref["y"], mag["y"], torch.float32, "y")
        close(g[j], ref["dx"], mag["dx"], torch.float32, "dx")


def test_in_place(sv):
    q, k = make(3, 77, 4, 64, torch.bfloat16, 3), make(4, 1234, 4, 64, torch.bfloat16, 3)
    freq = torch.logspace(0, -3, 24, dtype=torch.float64, device="cuda")
    kw = dict(wq=q["w"], wk=k["w"], axis_pairs=[8, 8, 8])
    want = sv.svconv_qk_norm_rope_fwd(q["x"], k["x"], q["pos"], k["pos"], freq, **kw)
    wg = sv.svconv_qk_norm_rope_bwd(q["dy"], k["dy"], q["x"], k["x"], q["pos"], k["pos"], freq, **kw)
    dq, dk = q["dy"].clone(), k["dy"].clone()
    g = sv.svconv_qk_norm_rope_bwd(dq, dk, q["x"], k["x"], q["pos"], k["pos"], freq, dQ=dq, dK=dk, **kw)
    a, b = q["x"].clone(), k["x"].clone()
    sv.svconv_qk_norm_rope_fwd(a, b, q["pos"], k["pos"], freq, Yq=a, Yk=b, **kw)
    torch.cuda.synchronize()
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    for u, v in zip(g, wg):
        assert torch.equal(u, v)


def test_gradients_against_differences(sv):
    q, k = make(5, 6, 2, 16, torch.float32, 2), make(6, 4, 1, 16, torch.float32, 2)
    freq = torch.logspace(0, -1, 8, dtype=torch.float64, device="cuda")
    g = sv.svconv_qk_norm_rope_bwd(q["dy"], k["dy"], q["x"], k["x"], q["pos"], k["pos"], freq, wq=q["w"], wk=k["w"], axis_pairs=[3, 5])
    for j, s in enumerate((q, k)):
        f = lambda t: float((reference(t, [3, 5], freq, "half", 1e-6)[0]["y"] * s["dy"].double()).sum())
        for name, got in (("x", g[j]), ("w", g[2 + j])):
            gen = torch.Generator().manual_seed(j)
            step = torch.randn(s[name].shape, generator=gen, dtype=torch.float64).cuda()
            up, dn = dict(s), dict(s)
            up[name], dn[name] = s[name].double() + 1e-6 * step, s[name].double() - 1e-6 * step
            slope = (f(up) - f(dn)) / 2e-6
            assert abs(slope - float((got.double() * step).sum())) <= 1e-5 * float((got.double().abs() * step.abs()).sum()) + 1e-6


def test_captured_graph(sv):
    q, k = make(7, 40, 4, 64, torch.bfloat16, 1), make(8, 900, 4, 64, torch.bfloat16, 1)
    freq = torch.logspace(0, -3, 32, dtype=torch.float64, device="cuda")
    args = (q["x"], k["x"], q["pos"], k["pos"], freq)
    want = sv.svconv_qk_norm_rope_fwd(*args) + sv.svconv_qk_norm_rope_bwd(q["dy"], k["dy"], *args)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = sv.svconv_qk_norm_rope_fwd(*args) + sv.svconv_qk_norm_rope_bwd(q["dy"], k["dy"], *args)
    for _ in range(2):
        gr.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("lo,hi", [(0, 282624), (2 ** 30, 2 ** 31 - 1)])
def test_fp32_angles_at_any_position(sv, layout, lo, hi):
    """(2, 0) turned by the angle, against the angle as a rational number of turns.  The norm of these rows is exactly 1,
    so the turned pair is off by the sine and cosine alone: one unit in the last place each (2^-24), an angle held in
    24 bits on an eighth of a turn either way (2^-27 of half a turn) and the turn's fraction in 32 bits.  In the mean
    square a rounding is 1 / sqrt(3) of its bound."""
    n, pairs, d = 500, 16, 32
    gen = torch.Generator(device="cuda")
    gen.manual_seed(lo % 1000)
    pos = torch.randint(lo, hi, (n,), generator=gen, device="cuda").int()
    pos[0], pos[1::2] = 0, -pos[1::2]
    x = torch.zeros((n, 1, d), device="cuda")
    a, b = (torch.arange(8), torch.arange(8) + pairs) if layout == "half" else (2 * torch.arange(8), 2 * torch.arange(8) + 1)
    x[..., a] = 2.0
    freq = (10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).cuda()
    empty = x[:0], pos[:0]
    y, _ = sv.svconv_qk_norm_rope_fwd(x, empty[0], pos, empty[1], freq, eps=0.0, layout=layout)
    assert (y[0, 0, a] == 2).all() and (y[0, 0, b] == 0).all()
    # turns = pos * freq / (2 pi) modulo 1, 1 / (2 pi) from pi = 16 atan(1/5) - 4 atan(1/239) in integers
    bits = 256
    def atan_inv(m):
        s, term, k = 0, (1 << bits) // m, 1
        while term:
            s += term // k if k % 4 == 1 else -(term // k)
            term, k = term // (m * m), k + 2
        return s
    two_pi = 2 * (16 * atan_inv(5) - 4 * atan_inv(239))
    off = []
    for i in range(8):
        num, den = float(freq[i]).as_integer_ratio()
        for p, ya, yb in zip(pos.tolist(), y[:, 0, a[i]].tolist(), y[:, 0, b[i]].tolist()):
            turns = (p * num << bits + 64) // (den * two_pi)  # units of 2^-64
            part = ((turns + (1 << 63)) % (1 << 64) - (1 << 63)) / 2.0 ** 64
            ang = 2 * math.pi * part
            off.append((yb * math.cos(ang) - ya * math.sin(ang)) / 2)
    rms = math.sqrt(sum(v * v for v in off) / len(off))
    bound = math.sqrt((2.0 ** -24) ** 2 + (math.pi * 2.0 ** -27) ** 2 + (2 * math.pi * 2.0 ** -32) ** 2) / math.sqrt(3)
    assert rms <= bound, (rms, bound)
