"""svconv_cross_attn_fwd / _bwd against the formulas in 64 bits.

Bounds, element by element.  A bf16 rounding is off by at most u = 2^-8 of the value.  Forward:
the weights P are rounded once as matrix operands and O once at the end, so |err| <= u (sum_j P |V|
+ |O|).  Backward: P and dS are rounded once each, D = dO . O takes the rounded O (off by at most
dD = u sum_c |dO| (|O| + sum_j P |V|)), and each gradient is rounded at the end:
    dV:  u (P^T |dO| + |dV|)
    dQ:  u (scale |dS| |K| + |dQ|) + scale (P dD) |K|,   dK the same with |Q| and the transposes.
5% on top covers the products of these terms and the fp32 sums; lse is an fp32 sum of fp32 scores,
whose d products each round by 2^-24 of their magnitude.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = torch.finfo(torch.bfloat16).eps / 2


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_convolution_pruned_b200 import build, svconv
    build.build()
    assert svconv.svconv_read_error_word() == 0
    return svconv


def offsets(lens, start=0):
    return torch.tensor(np.concatenate([[start], start + np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def make(seed, q_lens, kv_lens, Hq, Hkv, d, keep=1.0, gap=0, fused=False, scale=1.0):
    """Inputs with `gap` rows of no group before the first and after the last one."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    nq, nk = sum(q_lens) + 2 * gap, sum(kv_lens) + 2 * gap
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
    x = {"Q": (scale * rnd(nq, Hq, d)).bfloat16()}
    if fused:  # K and V as slices of one projection of [K | V | something else]
        kv = rnd(nk, 2 * Hkv + 1, d).bfloat16()
        x["K"], x["V"] = kv[:, :Hkv], kv[:, Hkv:2 * Hkv]
    else:
        x["K"], x["V"] = rnd(nk, Hkv, d).bfloat16(), rnd(nk, Hkv, d).bfloat16()
    x["dO"] = rnd(nq, Hq, d).bfloat16()
    x["q_off"], x["kv_off"] = offsets(q_lens, gap), offsets(kv_lens, gap)
    x["keep"] = (torch.rand((nk,), generator=gen, device="cuda") < keep).to(torch.uint8) if keep < 1 else None
    x["max_q"], x["max_kv"] = max(q_lens), max(kv_lens)
    return x


def reference(x, scale, O_used=None):
    """O, lse, dQ, dK, dV in fp64 with their bounds, group by group and head by head."""
    Q, K, V, dO = (x[k].double() for k in ("Q", "K", "V", "dO"))
    nq, Hq, d = Q.shape
    r = Hq // K.shape[1]
    z = lambda t: torch.zeros_like(t)
    out = {k: z(t) for k, t in (("O", Q), ("dQ", Q), ("dK", K), ("dV", V))}
    tol = {k: z(t) for k, t in out.items()}
    out["lse"] = torch.full((nq, Hq), -math.inf, dtype=torch.float64, device="cuda")
    tol["lse"] = torch.zeros((nq, Hq), dtype=torch.float64, device="cuda")
    qo, ko = x["q_off"].tolist(), x["kv_off"].tolist()
    for g in range(len(qo) - 1):
        a, b = torch.arange(qo[g], qo[g + 1], device="cuda"), torch.arange(ko[g], ko[g + 1], device="cuda")
        if x["keep"] is not None:
            b = b[x["keep"][b] != 0]
        if len(a) == 0 or len(b) == 0:
            continue
        for h in range(Hq):
            q, k, v, do = Q[a, h], K[b, h // r], V[b, h // r], dO[a, h]
            s = scale * q @ k.T
            lse = torch.logsumexp(s, 1, keepdim=True)
            P = torch.exp(s - lse)
            O, A = P @ v, P @ v.abs()
            out["O"][a, h], out["lse"][a, h] = O, lse[:, 0]
            tol["O"][a, h] = U * (A + O.abs())
            tol["lse"][a, h] = 2.0 ** -20 * (1 + lse[:, 0].abs()) + 2.0 ** -24 * (d + 8) * abs(scale) * (q.abs() @ k.abs().T).amax(1)
            dS = P * (do @ v.T - (do * O).sum(1, keepdim=True))
            slop = P * (U * (do.abs() * (O.abs() + A)).sum(1, keepdim=True))
            dq = scale * dS @ k
            out["dQ"][a, h] = dq
            tol["dQ"][a, h] = abs(scale) * (U * dS.abs() + slop) @ k.abs() + U * dq.abs()
            out["dK"][b, h // r] += scale * dS.T @ q
            tol["dK"][b, h // r] += abs(scale) * (U * dS.abs() + slop).T @ q.abs()
            out["dV"][b, h // r] += P.T @ do
            tol["dV"][b, h // r] += U * P.T @ do.abs()
    for k in ("dK", "dV"):
        tol[k] += U * out[k].abs()
    return out, tol


def close(got, ref, tol, what):
    got = got.double()
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), fin), f"{what}: finite in other places"
    assert torch.equal(got[~fin], ref[~fin]), what
    over = (got - ref).abs()[fin] - 1.05 * tol[fin] - 1e-30
    assert over.numel() == 0 or float(over.max()) <= 0, f"{what}: {float(over.max()):.3e} over its bound"


def run_both(sv, x, scale=None, backward=True, **kw):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dict(max_q=x["max_q"], max_kv=x["max_kv"], kv_keep=x["keep"], scale=scale, status=st)
    args.update(kw)
    sentinel = 7.0
    O = torch.full_like(x["Q"], sentinel)
    lse = torch.full(x["Q"].shape[:2], sentinel, device="cuda")
    sv.svconv_cross_attn_fwd(x["Q"], x["K"], x["V"], x["q_off"], x["kv_off"], out=O, lse=lse, **args)
    got = {"O": O, "lse": lse}
    if backward:
        dQ = torch.full_like(x["Q"], sentinel)
        dK, dV = (torch.full(x["K"].shape, sentinel, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        sv.svconv_cross_attn_bwd(x["dO"], x["Q"], x["K"], x["V"], O, lse, x["q_off"], x["kv_off"], dQ=dQ, dK=dK, dV=dV, **args)
        got.update(dQ=dQ, dK=dK, dV=dV)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and sv.svconv_read_error_word() == 0
    return got


def check(x, got, scale, what):
    ref, tol = reference(x, scale)
    spans = {"O": "q_off", "lse": "q_off", "dQ": "q_off", "dK": "kv_off", "dV": "kv_off"}
    for k, t in got.items():
        lo, hi = int(x[spans[k]][0]), int(x[spans[k]][-1])
        close(t[lo:hi], ref[k][lo:hi], tol[k][lo:hi], f"{what} {k}")
        for part in (t[:lo], t[hi:]):  # rows of no group are left as they were
            assert (part == 7.0).all(), f"{what}: {k} written outside the groups"


CASES = [
    # q lengths, kv lengths, Hq, Hkv, d, keep, gap, fused
    ((1,), (1,), 1, 1, 64, 1.0, 0, False),
    ((1,), (128,), 4, 4, 64, 1.0, 0, False),
    ((1, 1, 1), (129, 0, 257), 2, 1, 128, 1.0, 3, False),
    ((127, 128, 129), (127, 128, 129), 2, 2, 64, 1.0, 0, False),
    ((300, 0, 5, 64), (7, 40, 0, 500), 4, 2, 128, 1.0, 2, False),
    ((257,), (1000,), 3, 1, 64, 0.7, 0, False),
    ((33, 260), (129, 65), 5, 1, 96, 0.9, 1, True),
    ((65, 1), (3, 700), 6, 2, 40, 1.0, 0, True),
    ((40,), (90,), 2, 2, 8, 1.0, 5, False),
    ((90, 12), (17, 150), 2, 2, 24, 0.5, 0, False),
    ((70, 130), (300, 2), 4, 4, 80, 1.0, 0, True),
    ((520,), (640,), 1, 1, 16, 1.0, 0, False),
    ((3,), (5000,), 7, 7, 32, 0.95, 0, False),
    ((2, 30), (6000, 4100), 8, 1, 128, 1.0, 0, False),
    ((1100,), (30,), 2, 2, 72, 1.0, 0, False),
    ((385, 700), (513, 900), 2, 1, 128, 0.8, 0, False),
    ((20, 90), (60, 300), 64, 1, 64, 1.0, 0, False),
    ((37,), (200,), 21, 1, 128, 1.0, 0, False),
    ((1,), (20000,), 4, 4, 64, 1.0, 0, False),
    ((2300,), (100,), 4, 4, 64, 1.0, 0, False),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_against_the_formulas(sv, i):
    q_lens, kv_lens, Hq, Hkv, d, keep, gap, fused = CASES[i]
    x = make(100 + i, q_lens, kv_lens, Hq, Hkv, d, keep, gap, fused)
    got = run_both(sv, x)
    check(x, got, d ** -0.5, CASES[i])
    again = run_both(sv, x)
    for k in got:
        assert torch.equal(got[k], again[k]), f"{k} differs between two calls"


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_scales(sv, scale):
    x = make(7, (140, 3), (260, 31), 2, 2, 64)
    check(x, run_both(sv, x, scale=scale), scale, f"scale {scale}")


def test_strided_queries(sv):
    """Q as heads 1.. of a wider tensor; K and V as every other head of one."""
    x = make(6, (140, 3), (260, 31), 4, 2, 64)
    wide = torch.zeros((x["Q"].shape[0], 5, 64), dtype=torch.bfloat16, device="cuda")
    wide[:, 1:] = x["Q"]
    kv = torch.zeros((x["K"].shape[0], 4, 64), dtype=torch.bfloat16, device="cuda")
    kv[:, 0::2], kv[:, 1::2] = x["K"], x["V"]
    want = run_both(sv, x)
    y = dict(x, Q=wide[:, 1:], K=kv[:, 0::2], V=kv[:, 1::2])
    got = run_both(sv, y)
    for k in want:
        assert torch.equal(want[k], got[k]), k


def test_rows_beyond_32_bit_offsets(sv):
    """17 million keys of 128 channels: element offsets pass 2^31.  The mask keeps the last 900 and a few early ones."""
    n, d = 17_000_000, 128
    x = make(30, (5,), (900,), 1, 1, d)
    at = torch.cat([torch.arange(0, 300, device="cuda"), torch.arange(n - 600, n, device="cuda")])
    big = {k: torch.zeros((n, 1, d), dtype=torch.bfloat16, device="cuda") for k in ("K", "V")}
    for k in big:
        big[k][at] = x[k]
    keep = torch.zeros((n,), dtype=torch.uint8, device="cuda")
    keep[at] = 1
    y = dict(x, K=big["K"], V=big["V"], keep=keep, kv_off=offsets((n,)), max_kv=n)
    args = dict(max_q=5, max_kv=n, kv_keep=keep)
    O, lse = sv.svconv_cross_attn_fwd(y["Q"], y["K"], y["V"], y["q_off"], y["kv_off"], **args)
    dQ, dK, dV = sv.svconv_cross_attn_bwd(y["dO"], y["Q"], y["K"], y["V"], O, lse, y["q_off"], y["kv_off"], **args)
    torch.cuda.synchronize()
    check(x, {"O": O, "lse": lse, "dQ": dQ, "dK": dK[at], "dV": dV[at]}, d ** -0.5, "17M keys")
    assert not dK[300:n - 600].any() and not dV[300:n - 600].any()


FEW = [  # at most 32 query rows (tokens x heads of a key head) a group
    ((16, 16, 16, 16), (900, 1300, 1, 640), 4, 4, 64, 1.0, 0, False),
    ((32,), (5000,), 1, 1, 128, 1.0, 0, False),
    ((31, 0, 7), (300, 200, 0), 2, 2, 64, 0.7, 2, True),
    ((10, 3), (1000, 129), 3, 1, 96, 0.9, 1, False),
    ((1, 0, 1), (4000, 500, 127), 32, 1, 128, 0.5, 3, False),
    ((4, 2), (257, 3000), 24, 4, 40, 1.0, 0, True),
    ((5, 5, 5), (128, 128, 256), 5, 5, 8, 0.2, 0, False),
    ((2,) * 40, tuple(range(0, 400, 10)), 8, 2, 80, 0.9, 0, False),
    ((8, 1), (20000, 31), 4, 1, 64, 1.0, 0, False),
]


@pytest.mark.parametrize("i", range(len(FEW)))
def test_few_queries(sv, i):
    q_lens, kv_lens, Hq, Hkv, d, keep, gap, fused = FEW[i]
    x = make(60 + i, q_lens, kv_lens, Hq, Hkv, d, keep, gap, fused)
    got = run_both(sv, x)
    check(x, got, d ** -0.5, f"few queries {i}")
    again = run_both(sv, x)
    assert all(torch.equal(got[k], again[k]) for k in got)


FEW_KEYS = [  # at most 96 keys a group, more than 32 query rows
    ((700, 200), (77, 77), 4, 4, 64, 1.0, 0, False),
    ((500,), (96,), 2, 1, 128, 1.0, 0, False),
    ((300, 33, 0, 1), (1, 16, 17, 96), 2, 2, 64, 0.7, 2, True),
    ((130, 257, 40), (95, 0, 33), 3, 1, 96, 0.9, 1, False),
    ((40, 2), (5, 64), 32, 1, 128, 0.5, 3, False),
    ((1000, 43), (7, 12), 6, 2, 40, 0.5, 0, True),
    ((3000,), (30,), 1, 1, 8, 1.0, 0, False),
    (tuple(range(0, 200, 5)), (50,) * 40, 4, 2, 80, 0.9, 0, False),
    ((20000, 300), (65, 80), 2, 2, 64, 0.9, 4, False),
    ((9000,), (81,), 5, 1, 128, 1.0, 0, False),
]


@pytest.mark.parametrize("i", range(len(FEW_KEYS)))
def test_few_keys(sv, i):
    q_lens, kv_lens, Hq, Hkv, d, keep, gap, fused = FEW_KEYS[i]
    x = make(80 + i, q_lens, kv_lens, Hq, Hkv, d, keep, gap, fused)
    got = run_both(sv, x)
    check(x, got, d ** -0.5, f"few keys {i}")
    again = run_both(sv, x)
    assert all(torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("q_lens,kv_lens,H,d", [((13,), (107,), 4, 80), ((7, 7, 7), (22, 3, 9), 1, 32), ((6,) * 5, (3,) * 5, 2, 80),
                                                ((2, 30), (400, 200), 2, 128), ((100,), (64,), 2, 128)])
def test_few_rows_lose_nothing_but_the_last_rounding(sv, q_lens, kv_lens, H, d):
    """dS enters its products with 16 bits of significand, so dQ and dK are off by their own rounding: in norm at most
    u / sqrt(3) (a rounding is uniform within half a step), where one bf16 value for dS adds as much again.  D = dO . O with
    the rounded O adds a part of it that falls with the number of keys: 5%."""
    x = make(90 + d + H, q_lens, kv_lens, H, H, d)
    got = run_both(sv, x, backward=True)
    ref, _ = reference(x, d ** -0.5)
    for k in ("dQ", "dK"):
        off = float((got[k].double() - ref[k]).norm() / ref[k].norm())
        assert off <= 1.05 * U / math.sqrt(3), (k, off)


@pytest.mark.parametrize("d,Hq,Hkv", [(64, 2, 2), (128, 6, 2), (40, 1, 1)])
def test_a_single_key_has_no_score_gradient(sv, d, Hq, Hkv):
    """Groups of one key, or of one that is kept: weight 1 whatever the score, so dQ and dK are exactly 0."""
    x = make(79, (40, 7, 300), (1, 5, 1), Hq, Hkv, d)
    x["keep"] = torch.tensor([1, 0, 0, 0, 1, 0, 1], dtype=torch.uint8, device="cuda")
    got = run_both(sv, x)
    check(x, got, d ** -0.5, "single keys")
    assert (got["dQ"] == 0).all() and (got["dK"] == 0).all()


@pytest.mark.parametrize("d,Hq", [(64, 2), (128, 2), (64, 6), (128, 6)])
def test_few_keys_among_rows_that_hold_anything(sv, d, Hq):
    """The same as for few queries below, behind short key tiles and short last query tiles."""
    x = make(78, (95, 140), (30, 70), Hq, 2, d, keep=0.6, gap=9)
    want = run_both(sv, x)
    spoil(x)
    got = run_both(sv, x)
    for k in want:
        assert torch.equal(got[k], want[k]), k


def spoil(x):
    """NaN and infinities in dropped keys and in rows of no group."""
    qo, ko = x["q_off"].tolist(), x["kv_off"].tolist()
    out_q = torch.ones(x["Q"].shape[0], dtype=torch.bool, device="cuda")
    out_q[qo[0]:qo[-1]] = False
    drop = x["keep"] == 0
    drop[:ko[0]], drop[ko[-1]:] = True, True
    for n, k in enumerate(("K", "V")):
        x[k][drop] = float("nan") if n else float("inf")
    for k in ("Q", "dO"):
        x[k][out_q] = float("nan")


@pytest.mark.parametrize("d", [64, 128])
def test_few_queries_among_rows_that_hold_anything(sv, d):
    """NaN and infinities in dropped keys and in rows of other groups and of no group, behind short query tiles."""
    x = make(77, (5, 9), (300, 700), 2, 2, d, keep=0.6, gap=9)
    want = run_both(sv, x)
    spoil(x)
    got = run_both(sv, x)
    for k in want:
        assert torch.equal(got[k], want[k]), k


def test_many_groups(sv):
    """More groups than a warp has lanes, lengths from 0 on, some groups empty on either side."""
    rng = np.random.default_rng(5)
    q_lens, kv_lens = tuple(int(v) for v in rng.integers(0, 9, 150)), tuple(int(v) for v in rng.integers(0, 200, 150))
    x = make(31, q_lens, kv_lens, 4, 2, 64, keep=0.8, gap=2)
    check(x, run_both(sv, x), 0.125, "150 groups")
    x = make(32, (300,) * 40, (90,) * 40, 2, 1, 64)  # many items of one key tile each
    check(x, run_both(sv, x), 0.125, "40 groups")
    rng = np.random.default_rng(6)
    for d in (64, 128):  # more items than SMs, of none to three key tiles
        x = make(33, (300,) * 80, tuple(int(v) for v in rng.integers(0, 380, 80)), 4, 4, d, keep=0.9)
        check(x, run_both(sv, x), d ** -0.5, f"80 groups of {d} channels")


def test_large_scores_saturate_without_overflow(sv):
    """Scores of several hundred: the softmax collapses onto single keys."""
    x = make(8, (130,), (400,), 2, 2, 64, scale=60.0)
    check(x, run_both(sv, x), 64 ** -0.5, "saturated")


def test_rising_scores_move_the_running_maximum(sv):
    """Keys whose scores rise along the sequence: every key tile moves the maximum."""
    x = make(9, (150, 2), (1500, 2100), 2, 2, 64)
    for g in range(2):
        lo, hi = int(x["kv_off"][g]), int(x["kv_off"][g + 1])
        ramp = torch.linspace(-30.0, 30.0, hi - lo, device="cuda")
        x["K"][lo:hi, :, 0] = ramp[:, None].bfloat16()
    x["Q"][:, :, 0] = 8.0
    check(x, run_both(sv, x), 64 ** -0.5, "rising")


@pytest.mark.parametrize("d,lens", [(64, ((200, 40), (300, 150))), (128, ((3, 2), (900, 400)))])
def test_masked_and_foreign_rows_may_hold_anything(sv, d, lens):
    """NaN and infinities in dropped keys, and in rows of other groups and of no group."""
    x = make(11, lens[0], lens[1], 2, 2, d, keep=0.6, gap=9)
    ko, qo = x["kv_off"].tolist(), x["q_off"].tolist()
    x["keep"][ko[0] + 128:ko[0] + 256] = 0  # a whole tile of keys dropped
    clean = run_both(sv, x)
    check(x, clean, d ** -0.5, "clean")
    bad = torch.tensor([math.nan, math.inf, -math.inf], device="cuda").bfloat16()
    drop = (x["keep"] == 0).nonzero()[:, 0]
    for t in (x["K"], x["V"]):
        t[drop] = bad[torch.arange(len(drop), device="cuda") % 3][:, None, None]
        t[:ko[0]] = math.nan
        t[ko[-1]:] = math.inf
    for t in (x["Q"], x["dO"]):
        t[:qo[0]] = math.nan
        t[qo[-1]:] = math.inf
    dirty = run_both(sv, x)
    for k in clean:
        assert torch.equal(clean[k], dirty[k]), k
    # group 1 poisoned as a whole: group 0 keeps its values
    x["K"][ko[1]:], x["V"][ko[1]:], x["Q"][qo[1]:], x["dO"][qo[1]:] = math.nan, math.nan, math.nan, math.nan
    dirty = run_both(sv, x)
    for k, off in (("O", qo), ("lse", qo), ("dQ", qo), ("dK", ko), ("dV", ko)):
        assert torch.equal(clean[k][off[0]:off[1]], dirty[k][off[0]:off[1]]), k


def test_rows_without_any_key(sv):
    """A group whose mask drops every key, and one without keys: O = 0, lse = -inf, gradients 0."""
    x = make(12, (40, 30, 20), (200, 0, 10), 2, 1, 64, keep=0.5)
    x["keep"][:200] = 0
    got = run_both(sv, x)
    check(x, got, 0.125, "no keys")
    assert (got["O"][:70] == 0).all() and torch.isinf(got["lse"][:70]).all() and (got["dQ"][:70] == 0).all()
    assert (got["dK"][:200] == 0).all() and (got["dV"][:200] == 0).all()


def test_keys_without_queries_get_zero_gradients(sv):
    x = make(13, (0, 4), (300, 20), 2, 2, 64)
    got = run_both(sv, x)
    assert (got["dK"][:300] == 0).all() and (got["dV"][:300] == 0).all()
    check(x, got, 0.125, "no queries")


def test_gradients_against_differences(sv):
    """The backward pass against central differences of the fp64 forward formula."""
    x = make(14, (9, 5), (21, 12), 4, 2, 16)
    got = run_both(sv, x)
    ref, tol = reference(x, 0.25)
    f = lambda y: float((reference(y, 0.25)[0]["O"] * x["dO"].double()).sum())
    rng = np.random.default_rng(0)
    for name, grad in (("Q", "dQ"), ("K", "dK"), ("V", "dV")):
        step = torch.from_numpy(rng.standard_normal(tuple(x[name].shape))).cuda()
        eps = 1e-5
        up, dn = dict(x), dict(x)
        up[name], dn[name] = x[name].double() + eps * step, x[name].double() - eps * step
        slope = (f(up) - f(dn)) / (2 * eps)
        assert abs(slope - float((ref[grad] * step).sum())) <= 1e-6 * (1 + abs(slope))
        assert abs(slope - float((got[grad].double() * step).sum())) <= float((1.05 * tol[grad] * step.abs()).sum()) + 1e-5


def test_larger_groups_than_the_bound_are_flagged(sv):
    x = make(15, (40, 8), (300, 20), 2, 2, 64)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    full, _ = sv.svconv_cross_attn_fwd(x["Q"], x["K"], x["V"], x["q_off"], x["kv_off"], max_q=40, max_kv=300)
    O = torch.full_like(x["Q"], 7.0)
    sv.svconv_cross_attn_fwd(x["Q"], x["K"], x["V"], x["q_off"], x["kv_off"], max_q=16, max_kv=300, status=st, out=O)
    torch.cuda.synchronize()
    assert int(st.item()) == sv.STATUS_CHUNK_OVERFLOW
    assert torch.equal(O[:16], full[:16]) and (O[16:40] == 7.0).all() and torch.equal(O[40:], full[40:])


def test_bad_offsets_are_flagged_and_their_groups_skipped(sv):
    x = make(16, (40, 8), (300, 20), 2, 2, 64)
    want = run_both(sv, x)
    for bad in ([0, 300, 100000], [0, 300, 200], [-4, 300, 320]):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        g = 0 if bad[0] < 0 else 1
        O = torch.full_like(x["Q"], 7.0)
        lse = torch.full(x["Q"].shape[:2], 7.0, device="cuda")
        kw = dict(max_q=40, max_kv=300, status=st)
        sv.svconv_cross_attn_fwd(x["Q"], x["K"], x["V"], x["q_off"], off, out=O, lse=lse, **kw)
        dQ, dK, dV = torch.full_like(x["Q"], 7.0), torch.full_like(x["K"], 7.0), torch.full_like(x["V"], 7.0)
        sv.svconv_cross_attn_bwd(x["dO"], x["Q"], x["K"], x["V"], want["O"], want["lse"], x["q_off"], off, dQ=dQ,
                                 dK=dK, dV=dV, **kw)
        torch.cuda.synchronize()
        assert int(st.item()) == sv.STATUS_BAD_OFFSETS, bad
        good = slice(0, 40) if g == 1 else slice(40, 48)
        assert torch.equal(O[good], want["O"][good]) and torch.equal(dQ[good], want["dQ"][good])
        skipped = slice(40, 48) if g == 1 else slice(0, 40)
        assert (O[skipped] == 7.0).all() and (dQ[skipped] == 7.0).all() and (lse[skipped] == 7.0).all()
    assert sv.svconv_read_error_word() == 0


@pytest.mark.parametrize("q_lens,kv_lens", [((9, 8), (300, 20)), ((700, 600), (90, 20))])
def test_bad_offsets_and_bounds_with_few_rows(sv, q_lens, kv_lens):
    """The backward forms for few queries and for few keys: bad groups are skipped, rows past a bound left out."""
    x = make(17, q_lens, kv_lens, 2, 2, 64)
    want = run_both(sv, x)
    nq, nk = sum(q_lens), sum(kv_lens)

    def bwd(q_off, kv_off, max_q, max_kv):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = [torch.full_like(x[k], 7.0) for k in ("Q", "K", "V")]
        sv.svconv_cross_attn_bwd(x["dO"], x["Q"], x["K"], x["V"], want["O"], want["lse"], q_off, kv_off, max_q=max_q, max_kv=max_kv,
                                 status=st, dQ=out[0], dK=out[1], dV=out[2])
        torch.cuda.synchronize()
        return int(st.item()), out

    tens = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    a, b = q_lens[0], kv_lens[0]
    for q_off, kv_off in (([0, a, nq], [0, b, nk + 1]), ([0, a, a - 1], [0, b, nk])):
        flags, (dQ, dK, dV) = bwd(tens(q_off), tens(kv_off), max(q_lens), max(kv_lens))
        assert flags == sv.STATUS_BAD_OFFSETS
        assert torch.equal(dQ[:a], want["dQ"][:a]) and torch.equal(dK[:b], want["dK"][:b]) and torch.equal(dV[:b], want["dV"][:b])
        assert (dQ[a:] == 7.0).all() and (dK[b:] == 7.0).all() and (dV[b:] == 7.0).all()
    # a bound below the first group's keys, for the forward pass as well (a row's weights add up to 1 over the keys that
    # take part): the rest is not written, and the results are those of a mask over it
    short = b - 7
    y = dict(x)
    y["keep"] = torch.ones(nk, dtype=torch.uint8, device="cuda")
    y["keep"][short:b] = 0
    ref, tol = reference(y, 0.125)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    full = want
    want = dict(want)
    want["O"], want["lse"] = sv.svconv_cross_attn_fwd(x["Q"], x["K"], x["V"], x["q_off"], x["kv_off"], max_q=max(q_lens), max_kv=short,
                                                      status=st)
    flags, (dQ, dK, dV) = bwd(x["q_off"], x["kv_off"], max(q_lens), short)
    assert flags == sv.STATUS_CHUNK_OVERFLOW == int(st.item())
    assert (dK[short:b] == 7.0).all() and (dV[short:b] == 7.0).all()
    on = y["keep"] != 0
    for k, got in (("dK", dK[on]), ("dV", dV[on])):
        close(got, ref[k][on], tol[k][on], f"bounded {k}")
    close(dQ, ref["dQ"], tol["dQ"], "bounded dQ")
    want = full
    # a bound below the first group's queries
    if a > 8:
        flags, (dQ, dK, dV) = bwd(x["q_off"], x["kv_off"], a - 1, max(kv_lens))
        assert flags == sv.STATUS_CHUNK_OVERFLOW
        assert torch.equal(dQ[:a - 1], want["dQ"][:a - 1]) and (dQ[a - 1] == 7.0).all() and torch.equal(dQ[a:], want["dQ"][a:])
    assert sv.svconv_read_error_word() == 0


def test_streams_and_captured_graphs(sv):
    """A side stream, and two captured graphs (a workspace each) replayed on two streams."""
    xs = [make(20 + i, (33, 200), (2500, 700), 4, 2, 64) for i in range(2)]
    want = [run_both(sv, x) for x in xs]
    graphs, outs = [], []
    for x in xs:
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            run_both(sv, x)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            O, lse = sv.svconv_cross_attn_fwd(x["Q"], x["K"], x["V"], x["q_off"], x["kv_off"], max_q=200, max_kv=2500)
            d = sv.svconv_cross_attn_bwd(x["dO"], x["Q"], x["K"], x["V"], O, lse, x["q_off"], x["kv_off"], max_q=200,
                                         max_kv=2500)
        graphs.append((g, s))
        outs.append(dict(zip(("O", "lse", "dQ", "dK", "dV"), (O, lse) + d)))
    for _ in range(3):
        for g, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for k in w:
            assert torch.equal(o[k], w[k]), k
    assert sv.svconv_read_error_word() == 0


@pytest.mark.parametrize("q_lens,kv_lens", [((9, 8), (3000, 20)), ((2000, 600), (90, 20))])
def test_captured_backward_with_few_rows(sv, q_lens, kv_lens):
    """The backward forms for few queries and for few keys in a captured graph, replayed after the inputs changed."""
    x = make(18, q_lens, kv_lens, 2, 2, 64)
    kw = dict(max_q=max(q_lens), max_kv=max(kv_lens))

    def step():
        O, lse = sv.svconv_cross_attn_fwd(x["Q"], x["K"], x["V"], x["q_off"], x["kv_off"], **kw)
        return sv.svconv_cross_attn_bwd(x["dO"], x["Q"], x["K"], x["V"], O, lse, x["q_off"], x["kv_off"], **kw)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = step()
    for name in ("Q", "V", "dO"):
        x[name].mul_(-1.5)
        g.replay()
        torch.cuda.synchronize()
        want = run_both(sv, x)
        for k, t in zip(("dQ", "dK", "dV"), got):
            assert torch.equal(t, want[k]), (name, k)
    assert sv.svconv_read_error_word() == 0


@pytest.mark.parametrize("d,Hq,Hkv", [(128, 2, 2), (72, 6, 2)])
def test_wide_heads_backward_repeats_itself(sv, d, Hq, Hkv):
    """Above 64 channels the key pass keeps P and dS in the columns of the scores that two threads of a row read at their
    own pace: no timing may let one thread's results reach the other's scores."""
    x = make(140 + d, (1500, 700), (900, 1100), Hq, Hkv, d, keep=0.9)
    got = run_both(sv, x)
    check(x, got, d ** -0.5, f"{d} channels")
    args = dict(max_q=x["max_q"], max_kv=x["max_kv"], kv_keep=x["keep"])
    for _ in range(40):
        again = sv.svconv_cross_attn_bwd(x["dO"], x["Q"], x["K"], x["V"], got["O"], got["lse"], x["q_off"], x["kv_off"], **args)
        assert all(torch.equal(t, got[k]) for k, t in zip(("dQ", "dK", "dV"), again))


@pytest.mark.parametrize("d", [64, 128])
def test_short_items_one_after_the_other(sv, d):
    """Items of no key tile or one, whose loads are all issued before the rest of the CTA has its tensor memory, in
    calls that follow each other while the previous one's CTAs still hold theirs."""
    x = make(150 + d, (1, 3, 2, 5), (0, 7, 128, 90), 2, 1, d)
    got = run_both(sv, x, backward=False)
    check(x, got, d ** -0.5, f"short items of {d} channels")
    args = dict(max_q=x["max_q"], max_kv=x["max_kv"])
    outs = [sv.svconv_cross_attn_fwd(x["Q"], x["K"], x["V"], x["q_off"], x["kv_off"], **args) for _ in range(300)]
    torch.cuda.synchronize()
    assert all(torch.equal(O, got["O"]) and torch.equal(lse, got["lse"]) for O, lse in outs)
    assert sv.svconv_read_error_word() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_lens,kv_lens", [((3,), (9000,)), ((3000,), (90,)), ((260,), (20000,)), ((9000,), (260,))])
def test_workspaces_at_any_16_byte_boundary(sv, q_lens, kv_lens, d):
    """A caller's workspace of just the bytes asked for, 0 to 48 past a 512-byte boundary, between guards."""
    x = make(160 + d, q_lens, kv_lens, 2, 2, d)
    want = run_both(sv, x)
    _, desc = sv._attn_desc(x["Q"], x["K"], x["V"], x["q_off"], x["kv_off"], x["max_q"], x["max_kv"], None, None)
    sizes = sv.svconv_cross_attn_fwd_workspace_size(desc), sv.svconv_cross_attn_bwd_workspace_size(desc)
    assert max(sizes) > 0
    args = dict(max_q=x["max_q"], max_kv=x["max_kv"])
    for at in (0, 16, 32, 48):
        bufs = [torch.full((at + n + 64,), 0x55, dtype=torch.uint8, device="cuda") for n in sizes]
        fws, bws = (b[at:at + n] if n else None for b, n in zip(bufs, sizes))
        O, lse = sv.svconv_cross_attn_fwd(x["Q"], x["K"], x["V"], x["q_off"], x["kv_off"], workspace=fws, **args)
        grads = sv.svconv_cross_attn_bwd(x["dO"], x["Q"], x["K"], x["V"], O, lse, x["q_off"], x["kv_off"], workspace=bws, **args)
        torch.cuda.synchronize()
        for k, t in zip(("O", "lse", "dQ", "dK", "dV"), (O, lse) + grads):
            assert torch.equal(t, want[k]), (at, k)
        for b, n in zip(bufs, sizes):
            assert (b[:at] == 0x55).all() and (b[at + n:] == 0x55).all(), at
    assert sv.svconv_read_error_word() == 0


@pytest.mark.parametrize("q_lens,kv_lens,d,Hq", [
    ((200, 150), (300, 400), 64, 2), ((200, 150), (300, 400), 128, 4),      # two passes
    ((9, 5), (300, 700), 64, 2), ((3, 8), (20000, 300), 128, 4),            # few queries
    ((300, 40), (77, 90), 64, 4), ((20000, 700), (50, 64), 128, 2),         # few keys
])
def test_dropped_keys_get_zero_gradients_whatever_their_queries_hold(sv, q_lens, kv_lens, d, Hq):
    """A row of the group's own dO with an infinity, and one of Q with a NaN: a dropped key's gradients are 0 all the
    same, and rows and groups that do not meet those values keep theirs."""
    x = make(170 + d + Hq, q_lens, kv_lens, Hq, 2, d, keep=0.6)
    clean = run_both(sv, x)
    x["dO"][1, 0, 3] = math.inf
    x["Q"][2, Hq - 1, 5] = math.nan
    got = run_both(sv, x)
    drop = x["keep"] == 0
    assert drop.any()
    assert (got["dK"][drop] == 0).all() and (got["dV"][drop] == 0).all()
    rows = torch.ones(sum(q_lens), dtype=torch.bool, device="cuda")
    rows[1:3] = False
    for k in ("O", "lse", "dQ"):
        assert torch.equal(got[k][rows], clean[k][rows]), k
    for k in ("dK", "dV"):
        assert torch.equal(got[k][kv_lens[0]:], clean[k][kv_lens[0]:]), k
        assert not torch.isfinite(got[k][:kv_lens[0]][~drop[:kv_lens[0]]]).all()


@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv,d", [((13,), (77,), 4, 4, 80), ((13,), (96,), 4, 4, 80), ((8, 3), (70, 65), 2, 2, 128),
                                                     ((4, 2, 1), (90, 66, 80), 8, 1, 64)])
def test_few_queries_over_65_to_96_keys(sv, q_lens, kv_lens, Hq, Hkv, d):
    """At most 32 query rows: dS in 16 bits of significand there too, as over fewer or more keys (the bound of the test of
    norms above)."""
    x = make(180 + d, q_lens, kv_lens, Hq, Hkv, d)
    got = run_both(sv, x)
    check(x, got, d ** -0.5, "few by few")
    ref, _ = reference(x, d ** -0.5)
    for k in ("dQ", "dK"):
        off = float((got[k].double() - ref[k]).norm() / ref[k].norm())
        assert off <= 1.05 * U / math.sqrt(3), (k, off)
