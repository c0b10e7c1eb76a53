"""The operators in a run together: norm and rotation, cross-attention, their gradients, and the clipping of all
of them with a convolution's, against the same chain in 64 bits by autograd.

Bounds are norms: each bf16 tensor that passes from one operator to the next is off by u / sqrt(3) of its size at
most on average (u = 2^-8, a rounding is uniform within half a step), and so are the matrix operands P and dS.  A
gradient here passes at most eight such roundings (Yq, Yk, P, O, dS, dY, and its own, one of them twice), each at
most doubled by the terms it is a difference of: 16 u / sqrt(3) of its norm, 0.036.
"""
import math

import numpy as np
import pytest
import torch

from sparse_convolution_pruned_b200 import workloads as wl

pytestmark = pytest.mark.gpu
REL = 16 * 2.0 ** -8 / math.sqrt(3)


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_convolution_pruned_b200 import build, svconv
    build.build()
    return svconv


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def chain64(x, rot, q_lens, kv_lens, scale):
    """O by the formulas in fp64, differentiable."""
    def normed(t, pos, w):
        u = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + rot.eps) * w
        axis = torch.tensor([a for a, m in enumerate(rot.axis_pairs) for _ in range(m)], device="cuda")
        ang = (pos.double()[:, axis] * rot.freq)[:, None]
        p = len(rot.freq)
        a, b = u[..., :p], u[..., p:2 * p]
        return torch.cat([a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos(), u[..., 2 * p:]], -1)
    Yq, Yk = normed(x["Q"], x["pos_q"], x["wq"]), normed(x["K"], x["pos_k"], x["wk"])
    r = Yq.shape[1] // Yk.shape[1]
    out, q0, k0 = [], 0, 0
    for a, b in zip(q_lens, kv_lens):
        q, k, v = Yq[q0:q0 + a].transpose(0, 1), Yk[k0:k0 + b].transpose(0, 1), x["V"][k0:k0 + b].transpose(0, 1)
        k, v = k.repeat_interleave(r, 0), v.repeat_interleave(r, 0)
        out.append((torch.softmax(scale * q @ k.transpose(1, 2), -1) @ v).transpose(0, 1))
        q0, k0 = q0 + a, k0 + b
    return torch.cat(out)


@pytest.mark.parametrize("d,Hq,Hkv", [(64, 4, 4), (128, 4, 2)])
def test_chain_forward_backward_clip(sv, d, Hq, Hkv):
    from sparse_convolution_pruned_b200 import data_parallel, recombine as rc
    w = wl.custom_conv(seed=5, T=12, H=16, W=16, keep_frac=0.3, Cin=64, Cout=64, dtype="bf16")
    dev = lambda a, dt=None: (torch.from_numpy(np.ascontiguousarray(a)).to(dt) if dt else torch.from_numpy(np.ascontiguousarray(a))).cuda()
    coords, off = dev(w.coords), w.frame_off.astype(np.int64)
    # the keys are the sparse tokens, four frames to a group; the queries a few auxiliary tokens of each group
    kv_lens = [int(off[t + 4] - off[t]) for t in range(0, 12, 4)]
    q_lens = [3, 17, 150]
    nq, nk = sum(q_lens), sum(kv_lens)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(d)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
    x = {"Q": rnd(nq, Hq, d).bfloat16(), "K": rnd(nk, Hkv, d).bfloat16(), "V": rnd(nk, Hkv, d).bfloat16(),
         "wq": 1 + 0.2 * rnd(d), "wk": 1 + 0.2 * rnd(d), "pos_k": coords,
         "pos_q": torch.randint(0, 12, (nq, 3), generator=gen, device="cuda", dtype=torch.int32)}
    dO = rnd(nq, Hq, d).bfloat16()
    cum = lambda v: torch.tensor(np.concatenate([[0], np.cumsum(v)]), dtype=torch.int32, device="cuda")
    groups = rc.Groups(cum(q_lens), cum(kv_lens), max(q_lens), max(kv_lens))
    pairs = (d // 8, d // 8, d // 8)
    rot = rc.Rotation(rc.axis_frequencies(pairs, 100.0), pairs)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        nbr, _ = sv.svconv_build_index(coords, dev_off, w.T, w.H, w.W)
        dX, dW, db = sv.svconv_bwd(dY, X, nbr, Wt)
        O, saved = rc.recombine_fwd(x["Q"], x["K"], x["V"], x["pos_q"], x["pos_k"], groups, rot, wq=x["wq"], wk=x["wk"], status=st)
        g = rc.recombine_bwd(dO, saved, groups, rot, status=st)
        return O, (dW, db) + g

    dev_off, X, Wt, dY = dev(w.frame_off), dev(w.X, torch.bfloat16), dev(w.Wt, torch.bfloat16), dev(w.dY, torch.bfloat16)
    O, grads = step()
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and sv.svconv_read_error_word() == 0

    ref = {k: (v.double().requires_grad_(True) if v.is_floating_point() else v) for k, v in x.items()}
    O64 = chain64(ref, rot, q_lens, kv_lens, d ** -0.5)
    O64.backward(dO.double())
    assert rel(O, O64.detach()) <= REL
    names = ("dQ", "dK", "dV", "dwq", "dwk")
    for name, got, leaf in zip(names, grads[2:], ("Q", "K", "V", "wq", "wk")):
        assert rel(got, ref[leaf].grad) <= REL, name

    # clipping of everything together
    total = math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))
    keep = [g.clone() for g in grads]
    norm = data_parallel.allreduce_and_clip(grads, total / 5)
    torch.cuda.synchronize()
    assert abs(float(norm) - total) <= 2.0 ** -22 * total
    for g, k in zip(grads, keep):
        u = torch.finfo(g.dtype).eps / 2
        want = k.double() / 5
        assert ((g.double() - want).abs() <= (u + 2.0 ** -20) * want.abs() + 1e-38).all()

    # the whole step captured, replayed after its inputs changed
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=s):
        O2, grads2 = step()
        norm2 = data_parallel.allreduce_and_clip(grads2, total / 5)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(O2, O) and torch.equal(norm2, norm)
    for a, b in zip(grads2, grads):
        assert torch.equal(a, b)
    x["Q"].mul_(2.0)  # the norm takes a factor out again: O must not move beyond rounding
    gr.replay()
    torch.cuda.synchronize()
    assert rel(O2, O64.detach()) <= REL


def test_rotation_sees_relative_positions_only(sv):
    """Moving every position of both streams by the same offset leaves O where it was, within rounding."""
    from sparse_convolution_pruned_b200 import recombine as rc
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
    Q, K, V = rnd(40, 2, 64).bfloat16(), rnd(500, 2, 64).bfloat16(), rnd(500, 2, 64).bfloat16()
    pq = torch.randint(0, 500, (40,), generator=gen, device="cuda", dtype=torch.int32)
    pk = torch.arange(500, dtype=torch.int32, device="cuda")
    off = lambda n: torch.tensor([0, n], dtype=torch.int32, device="cuda")
    groups, rot = rc.Groups(off(40), off(500), 40, 500), rc.Rotation(rc.axis_frequencies((32,)), (32,))
    a, _ = rc.recombine_fwd(Q, K, V, pq, pk, groups, rot)
    b, _ = rc.recombine_fwd(Q, K, V, pq + 1_000_000, pk + 1_000_000, groups, rot)
    torch.cuda.synchronize()
    assert rel(a, b.double()) <= REL


def test_padded_batch(sv):
    """Rows behind the last group: zero gradients there, and the weights' gradients are those of the rows before."""
    from sparse_convolution_pruned_b200 import recombine as rc
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
    Q, K, V, dO = rnd(90, 4, 64).bfloat16(), rnd(400, 2, 64).bfloat16(), rnd(400, 2, 64).bfloat16(), rnd(90, 4, 64).bfloat16()
    wq, wk = 1 + 0.2 * rnd(64), 1 + 0.2 * rnd(64)
    pq, pk = torch.arange(90, dtype=torch.int32, device="cuda"), torch.arange(400, dtype=torch.int32, device="cuda")
    off = lambda *n: torch.tensor(n, dtype=torch.int32, device="cuda")
    groups, rot = rc.Groups(off(0, 20, 70), off(0, 110, 310), 50, 200), rc.Rotation(rc.axis_frequencies((32,)), (32,))

    def grads(nq, nk):
        _, saved = rc.recombine_fwd(Q[:nq], K[:nk], V[:nk], pq[:nq], pk[:nk], groups, rot, wq=wq, wk=wk)
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(4)]  # what memory may hold
        del junk
        return rc.recombine_bwd(dO[:nq], saved, groups, rot)

    exact, padded = grads(70, 310), grads(90, 400)
    torch.cuda.synchronize()
    for a, b in zip(exact[:3], padded[:3]):
        assert torch.equal(a, b[:len(a)]) and (b[len(a):] == 0).all()
    for a, b in zip(exact[3:], padded[3:]):  # the same terms and zeros, summed in another order
        assert rel(b, a.double()) <= REL


def test_scratch_of_a_call_on_another_stream(sv, monkeypatch):
    """Scratch memory that a call allocates is not given out again while its stream has the call before it."""
    taken = []
    scratch = sv._scratch

    def spy(*args):
        got = scratch(*args)
        taken.append(got[1:])
        return got
    monkeypatch.setattr(sv, "_scratch", spy)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
    off = lambda n: torch.tensor([0, n], dtype=torch.int32, device="cuda")
    Q, K, V = rnd(3, 2, 64).bfloat16(), rnd(9000, 2, 64).bfloat16(), rnd(9000, 2, 64).bfloat16()
    lim, g = dict(max_q=3, max_kv=9000), rnd(5000)
    pos, freq = (torch.arange(n, dtype=torch.int32, device="cuda") for n in (3, 9000)), torch.ones(32, dtype=torch.float64, device="cuda")
    pq, pk = pos
    calls = [
        lambda s: sv.svconv_cross_attn_fwd(Q, K, V, off3, off9, stream=s, **lim),
        lambda s: sv.svconv_cross_attn_bwd(Q, Q, K, V, O, lse, off3, off9, stream=s, **lim),
        lambda s: sv.svconv_qk_norm_rope_bwd(Q, K, Q, K, pq, pk, freq, stream=s),
        lambda s: sv.svconv_clip_grads([g], 1.0, stream=s),
    ]
    off3, off9 = off(3), off(9000)
    O, lse = sv.svconv_cross_attn_fwd(Q, K, V, off3, off9, **lim)
    side = torch.cuda.Stream()
    for call in calls:
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        del taken[:]
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)  # ~0.1 s
        call(side)
        (address, size), = taken
        assert size > 0
        fresh = [torch.empty((size,), dtype=torch.uint8, device="cuda") for _ in range(4)]
        assert all(t.data_ptr() != address for t in fresh)
    torch.cuda.synchronize()
    assert sv.svconv_read_error_word() == 0


def stream_calls(sv):
    """Every call that allocates, as call(stream) -> its outputs."""
    from sparse_convolution_pruned_b200 import recombine as rc
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
    off = lambda n: torch.tensor([0, n], dtype=torch.int32, device="cuda")
    Q, K, V = rnd(40, 2, 64).bfloat16(), rnd(9000, 2, 64).bfloat16(), rnd(9000, 2, 64).bfloat16()
    pq, pk = (torch.arange(n, dtype=torch.int32, device="cuda") for n in (40, 9000))
    groups, rot = rc.Groups(off(40), off(9000), 40, 9000), rc.Rotation(rc.axis_frequencies((32,)), (32,))
    lim, g = dict(max_q=40, max_kv=9000), [rnd(50000), rnd(7).bfloat16()]
    O, lse = sv.svconv_cross_attn_fwd(Q, K, V, groups.q_off, groups.kv_off, **lim)
    _, saved = rc.recombine_fwd(Q, K, V, pq, pk, groups, rot)
    torch.cuda.synchronize()
    return [
        lambda s: sv.svconv_cross_attn_fwd(Q, K, V, groups.q_off, groups.kv_off, stream=s, **lim),
        lambda s: sv.svconv_cross_attn_bwd(Q, Q, K, V, O, lse, groups.q_off, groups.kv_off, stream=s, **lim),
        lambda s: sv.svconv_qk_norm_rope_fwd(Q, K, pq, pk, rot.freq, stream=s),
        lambda s: sv.svconv_qk_norm_rope_bwd(Q, K, Q, K, pq, pk, rot.freq, stream=s),
        lambda s: (sv.svconv_clip_grads(g, math.inf, stream=s),),
        lambda s: rc.recombine_fwd(Q, K, V, pq, pk, groups, rot, stream=s)[:1],
        lambda s: rc.recombine_bwd(Q, saved, groups, rot, stream=s),
    ]


def spied(sv, monkeypatch):
    """The memory that calls allocate, as a list of (address, bytes)."""
    taken = []
    new = sv._new

    def spy(*args, **kw):
        t = new(*args, **kw)
        taken.append((t.data_ptr(), t.numel() * t.element_size()))
        return t
    monkeypatch.setattr(sv, "_new", spy)
    return taken


def overlaps(a, b):
    return any(x < v + n and v < x + m for x, m in a for v, n in b)


def test_dropped_results_of_a_call_on_another_stream(sv, monkeypatch):
    """What a call on another stream allocated and its caller dropped is not given out on the current stream while the
    call has yet to write it."""
    calls, taken, side = stream_calls(sv), spied(sv, monkeypatch), torch.cuda.Stream()
    for i, call in enumerate(calls):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        del taken[:]
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)  # ~0.1 s
        got = [(t.data_ptr(), t.numel() * t.element_size()) for t in call(side)]  # dropped at once
        used = taken + got
        fresh = [torch.empty((n,), dtype=torch.uint8, device="cuda") for _ in range(4) for _, n in used]
        assert not overlaps(used, [(t.data_ptr(), t.numel()) for t in fresh]), i
        del fresh
    torch.cuda.synchronize()
    assert sv.svconv_read_error_word() == 0


def test_two_calls_at_once_on_two_streams(sv, monkeypatch):
    """A call on the current stream that has not run yet, and the same call on another stream: no memory in common, and
    the results of calls one after the other."""
    calls, side = stream_calls(sv), torch.cuda.Stream()
    want = [[t.clone() for t in call(None)] for call in calls]
    taken = spied(sv, monkeypatch)
    for i, call in enumerate(calls):
        torch.cuda.synchronize()
        del taken[:]
        torch.cuda._sleep(200_000_000)
        first = call(torch.cuda.current_stream())
        mine = list(taken)
        del taken[:]
        second = call(side)
        assert mine and not overlaps(mine, taken), i
        assert not overlaps([(t.data_ptr(), t.numel() * t.element_size()) for t in first],
                            [(t.data_ptr(), t.numel() * t.element_size()) for t in second]), i
        torch.cuda.synchronize()
        for got in (first, second):
            assert all(torch.equal(a, b) for a, b in zip(got, want[i])), i
    assert sv.svconv_read_error_word() == 0


def test_another_stream_under_a_captured_graph(sv):
    """Calls on a stream that joins the capture of the current one."""
    calls = stream_calls(sv)
    want = [[t.clone() for t in call(None)] for call in calls]
    torch.cuda.synchronize()
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        side.wait_stream(main)
        got = [call(side) for call in calls]
        main.wait_stream(side)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("d", [64, 128])
def test_short_attention_and_convolutions_in_turn(sv, d):
    """Kernels that follow each other closely and all use tensor memory: the results of calls with waits between them."""
    w = wl.custom_conv(seed=6, T=6, H=16, W=16, keep_frac=0.3, Cin=64, Cout=64, dtype="bf16")
    dev = lambda a, dt=None: torch.from_numpy(np.ascontiguousarray(a)).to(dt).cuda() if dt else torch.from_numpy(np.ascontiguousarray(a)).cuda()
    X, Wt, coords, foff = dev(w.X, torch.bfloat16), dev(w.Wt, torch.bfloat16), dev(w.coords), dev(w.frame_off)
    nbr, _ = sv.svconv_build_index(coords, foff, w.T, w.H, w.W)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
    off = lambda *n: torch.tensor(n, dtype=torch.int32, device="cuda")
    Q, K, V = rnd(200, 2, d).bfloat16(), rnd(300, 2, d).bfloat16(), rnd(300, 2, d).bfloat16()
    qo, ko = off(0, 2, 2, 200), off(0, 1, 120, 300)
    step = lambda: (sv.svconv_fwd(X, nbr, Wt), *sv.svconv_cross_attn_fwd(Q, K, V, qo, ko, max_q=198, max_kv=180))
    want = []
    for t in step():
        torch.cuda.synchronize()
        want.append(t.clone())
    got = [step() for _ in range(200)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    assert sv.svconv_read_error_word() == 0


def test_convolution_calls_on_another_stream(sv, monkeypatch):
    """The two tests above for the convolution, the adapter and the attention of auxiliary tokens."""
    w = wl.custom_conv(seed=8, T=8, H=16, W=16, keep_frac=0.4, Cin=64, Cout=64, dtype="bf16")
    dev = lambda a, dt=None: torch.from_numpy(np.ascontiguousarray(a)).to(dt).cuda() if dt else torch.from_numpy(np.ascontiguousarray(a)).cuda()
    X, Wt, dY = (dev(a, torch.bfloat16) for a in (w.X, w.Wt, w.dY))
    coords, foff = dev(w.coords), dev(w.frame_off)
    nbr, _ = sv.svconv_build_index(coords, foff, w.T, w.H, w.W)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(9)
    rnd = lambda *s: (0.1 * torch.randn(s, generator=gen, device="cuda")).bfloat16()
    rows = int(np.diff(w.frame_off).max()) * 4
    H, Wd, Wc, Wu, aux = rnd(w.n, 128), rnd(64, 128), rnd(64, 9, 64), rnd(128, 64), rnd(1, 4, 64)
    goff = torch.tensor([0, w.n], dtype=torch.int32, device="cuda")
    calls = [
        lambda s: sv.svconv_build_index(coords, foff, w.T, w.H, w.W, want_map=True, stream=s),
        lambda s: (sv.svconv_fwd(X, nbr, Wt, stream=s), sv.svconv_bwd_data(dY, nbr, Wt, stream=s)),
        lambda s: sv.svconv_bwd_weight(dY, X, nbr, stream=s),
        lambda s: sv.svconv_bwd(dY, X, nbr, Wt, stream=s),
        lambda s: sv.svconv_bwd_single_pass(dY, X, nbr, Wt, stream=s),
        lambda s: (sv.svconv_xattn_aux(X, goff, aux, max_group_rows=w.n, stream=s),),
    ]
    adapter = lambda Y, s: sv.svconv_adapter_fwd_xattn(Y, nbr, foff, w.T, Wd, Wc, Wu, aux[0], chunk_T=4, max_chunk_rows=rows, stream=s)
    want = [[t.clone() for t in call(None)] for call in calls] + [[t.clone() for t in adapter(H.clone(), None)]]
    torch.cuda.synchronize()
    taken, side = spied(sv, monkeypatch), torch.cuda.Stream()
    for i in range(len(want)):
        call = calls[i] if i < len(calls) else lambda s: adapter(Y if s is side else H.clone(), s)
        Y = H.clone()
        torch.cuda.synchronize()
        del taken[:]
        torch.cuda._sleep(200_000_000)
        first, mine = call(torch.cuda.current_stream()), list(taken)
        del taken[:]
        second = call(side)
        assert taken and not overlaps(mine, taken), i
        torch.cuda.synchronize()
        for got in (first, second):
            assert all(torch.equal(a, b) for a, b in zip(got, want[i])), i
        first = second = got = None
        Y = H.clone()
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        del taken[:]
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)
        call(side)  # dropped at once
        fresh = [torch.empty((n,), dtype=torch.uint8, device="cuda") for _ in range(4) for _, n in taken]
        assert not overlaps(taken, [(t.data_ptr(), t.numel()) for t in fresh]), i
        del fresh
    torch.cuda.synchronize()
    assert sv.svconv_read_error_word() == 0
