"""svconv_clip_grads against the definition in 64 bits.

Bounds: the squares are summed in fp64, so the norm is off by its own fp32 rounding (2^-24); the
factor adds three fp32 roundings and the product one more of the gradient's type.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_convolution_pruned_b200 import build, svconv
    build.build()
    return svconv


def make(seed, sizes, dtypes=(torch.float32,), scale=1.0, shift=0):
    """Gradients as views of flat buffers, each starting `shift` values off a 16-byte boundary at least."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    grads = []
    for i, n in enumerate(sizes):
        dt = dtypes[i % len(dtypes)]
        grads.append((scale * torch.randn((n + shift,), generator=gen, device="cuda")).to(dt)[shift:])
    return grads


def norm_of(grads):
    return math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))


def check(out, grads, max_norm, norm, what=""):
    ref = norm_of(grads)
    assert abs(float(norm) - ref) <= 2.0 ** -23 * ref, what
    f = min(1.0, max_norm / (ref + 1e-6))
    for o, g in zip(out, grads):
        r = g.double() * f
        u = torch.finfo(g.dtype).eps / 2
        assert ((o.double() - r).abs() <= (u + 2.0 ** -21) * r.abs() + torch.finfo(g.dtype).tiny * 2 ** -6).all(), what


SIZES = [
    ([1], 0), ([3, 0, 5], 0), ([64, 16], 1), ([8192, 8191, 8193, 1], 0), ([1000003], 3),
    ([147456, 64] * 20, 0), ([33 * 7] * 300, 0), ([5] * 1700, 2), ([3_000_000, 17, 2_000_001], 1),
]


@pytest.mark.parametrize("i", range(len(SIZES)))
@pytest.mark.parametrize("kind", ["f32", "bf16", "both"])
def test_norm_and_clipping(sv, i, kind):
    sizes, shift = SIZES[i]
    dts = {"f32": (torch.float32,), "bf16": (torch.bfloat16,), "both": (torch.float32, torch.bfloat16)}[kind]
    grads = make(i, sizes, dts, shift=shift)
    total = norm_of(grads)
    for max_norm in (total / 3, total * 3, math.inf, 0.0):
        out = [torch.empty_like(g) for g in grads]
        norm = sv.svconv_clip_grads(grads, max_norm, out=out)
        check(out, grads, max_norm, norm, (sizes[:4], kind, max_norm))
    keep = [g.clone() for g in grads]
    norm = sv.svconv_clip_grads(grads, total / 3)  # in place
    again = [torch.empty_like(g) for g in grads]
    norm2 = sv.svconv_clip_grads(keep, total / 3, out=again)
    assert torch.equal(norm, norm2)
    for a, b in zip(grads, again):
        assert torch.equal(a, b)


def test_misaligned_outputs_and_neighbours_are_left_alone(sv):
    """Outputs that start off a boundary differently from their inputs, with guards around them."""
    g = make(4, [5000, 777])
    for shift in range(4):
        buf = torch.full((6000,), 9.0, device="cuda")
        out = [buf[shift:shift + 5000], buf[5001 + shift:5778 + shift]]
        check(out, g, 1.0, sv.svconv_clip_grads(g, 1.0, out=out))
        rest = torch.cat([buf[:shift], buf[shift + 5000:shift + 5001], buf[shift + 5778:]])
        assert (rest == 9.0).all()


def test_norm_does_not_overflow_and_keeps_small_values(sv):
    for scale in (1e25, 1e-25):
        g = make(5, [100000, 33], scale=scale)
        total = norm_of(g)
        out = [torch.empty_like(x) for x in g]
        norm = sv.svconv_clip_grads(g, total / 2, out=out)
        assert abs(float(norm) - total) <= 2.0 ** -23 * total
        if scale > 1:
            check(out, g, total / 2, norm)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_gradients_that_are_not_finite_pass_unscaled(sv, bad):
    g = make(6, [9000, 50])
    g[1][7] = bad
    keep = [x.clone() for x in g]
    norm = sv.svconv_clip_grads(g, 0.5)
    assert not math.isfinite(float(norm))
    for a, b in zip(g, keep):
        assert torch.equal(a.nan_to_num(nan=5.0), b.nan_to_num(nan=5.0))


def test_zero_and_no_gradients(sv):
    z = [torch.zeros(100, device="cuda"), torch.zeros(0, device="cuda")]
    assert float(sv.svconv_clip_grads(z, 1.0)) == 0.0 and (z[0] == 0).all()
    norm = torch.full((), 3.0, device="cuda")
    assert float(sv.svconv_clip_grads([], 1.0, norm=norm)) == 0.0


def test_captured_graph_and_side_stream(sv):
    g = make(7, [147456, 64, 33])
    out = [torch.empty_like(x) for x in g]
    want = [torch.empty_like(x) for x in g]
    n0 = sv.svconv_clip_grads(g, 1.0, out=want)
    torch.cuda.synchronize()
    gr, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(gr, stream=s):
        n1 = sv.svconv_clip_grads(g, 1.0, out=out)
    for _ in range(3):
        gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(n0, n1) and all(torch.equal(a, b) for a, b in zip(out, want))
