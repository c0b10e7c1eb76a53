"""Refusals of the cross-attention, query/key norm and clipping entry points: all host checks,
made before any device call (no GPU needed)."""
import ctypes
import math

import pytest

from sparse_convolution_pruned_b200 import build as svbuild
from sparse_convolution_pruned_b200 import svconv as sv

NULL, SIZE, UNSUP, ALIGN, WORKSPACE = -1, -2, -3, -4, -5
P = ctypes.c_void_p
A = P(0x10000)     # an aligned address that no call may read
ODD = P(0x10008)


@pytest.fixture(scope="module")
def L():
    svbuild.build()
    return sv.lib()


def desc(**kw):
    c = dict(nq=8, nkv=16, Hq=4, Hkv=2, d=64, G=1, q_off=0x10000, kv_off=0x10000, max_q=8, max_kv=16, kv_keep=None,
             scale=0.125, q_row=256, q_head=64, k_row=128, k_head=64, v_row=128, v_head=64)
    c.update(kw)
    return sv.CrossAttnDesc(*[c[f] for f, _ in sv.CrossAttnDesc._fields_])


def fwd(L, d, Q=A, K=A, V=A, O=A, lse=A, ws=A, n=1 << 40):
    return L.svconv_cross_attn_fwd(ctypes.byref(d) if d is not None else None, Q, K, V, O, lse, ws, n, None, None)


def bwd(L, d, dO=A, Q=A, K=A, V=A, O=A, lse=A, dQ=A, dK=A, dV=A, ws=A, n=1 << 40):
    return L.svconv_cross_attn_bwd(ctypes.byref(d) if d is not None else None, dO, Q, K, V, O, lse, dQ, dK, dV, ws, n, None, None)


@pytest.mark.parametrize("bad,code", [
    (dict(nq=-1), SIZE), (dict(nkv=-1), SIZE), (dict(nq=2**31 - 1), SIZE), (dict(nkv=2**31 - 1), SIZE), (dict(G=-1), SIZE), (dict(max_q=-1), SIZE), (dict(max_kv=-1), SIZE),
    (dict(Hq=2**16, Hkv=2**16), SIZE), (dict(G=2**16), SIZE),
    (dict(Hq=0), SIZE), (dict(Hkv=0), SIZE), (dict(scale=math.nan), SIZE), (dict(scale=math.inf), SIZE),
    (dict(d=0), UNSUP), (dict(d=60), UNSUP), (dict(d=136), UNSUP), (dict(Hq=5), UNSUP), (dict(Hq=130, Hkv=2), UNSUP),
    (dict(q_off=None), NULL), (dict(kv_off=None), NULL),
    (dict(q_row=252), ALIGN), (dict(k_head=60), ALIGN), (dict(v_row=0), ALIGN), (dict(k_row=-128), ALIGN),
])
def test_cross_attention_descriptors(L, bad, code):
    assert fwd(L, desc(**bad)) == code
    assert bwd(L, desc(**bad)) == code


def test_cross_attention_arguments(L):
    assert fwd(L, None) == NULL and bwd(L, None) == NULL
    for name in ("Q", "K", "V", "O", "lse"):
        assert fwd(L, desc(), **{name: None}) == NULL, name
    for name in ("Q", "K", "V", "O"):
        assert fwd(L, desc(), **{name: ODD}) == ALIGN, name
    for name in ("dO", "Q", "K", "V", "O", "lse", "dQ", "dK", "dV"):
        assert bwd(L, desc(), **{name: None}) == NULL, name
    for name in ("dO", "Q", "K", "V", "O", "dQ", "dK", "dV", "ws"):
        assert bwd(L, desc(), **{name: ODD}) == ALIGN, name
    more = desc(nq=80, max_q=80, nkv=200, max_kv=200)  # beyond one tile of either side: statistics of every row
    need = L.svconv_cross_attn_bwd_workspace_size(ctypes.byref(more))
    assert need >= 80 * 4 * 4
    assert bwd(L, more, ws=None) == WORKSPACE and bwd(L, more, n=need - 1) == WORKSPACE
    many = desc(nkv=30000, max_kv=30000)  # few queries: splits of the keys
    need = L.svconv_cross_attn_bwd_workspace_size(ctypes.byref(many))
    assert need > 0 and bwd(L, many, n=need - 1) == WORKSPACE
    # nothing to do: accepted without pointers
    assert fwd(L, desc(G=0, q_off=None, kv_off=None), Q=None, O=None) == 0
    assert fwd(L, desc(max_q=0), Q=None, O=None) == 0
    assert bwd(L, desc(nq=0, nkv=0), dO=None, Q=None, K=None) == 0
    assert L.svconv_cross_attn_fwd_workspace_size(None) == 0 and L.svconv_cross_attn_bwd_workspace_size(None) == 0
    assert L.svconv_cross_attn_bwd_workspace_size(ctypes.byref(desc(d=60))) == 0


def side(**kw):
    c = dict(x=0x10000, x_row=256, n=8, H=4, pos=0x10000, w=None, y=0x20000, dy=0x10000, dx=0x10000, dw=0x10000)
    c.update(kw)
    return sv.QkSide(*[c[f] for f, _ in sv.QkSide._fields_])


def qk(L, dtype=sv.BF16, d=64, rot=32, layout=0, freq=A, axes=1, split=(16,), eps=1e-6, q=None, k=None, bwd=False, ws=A, n=1 << 30):
    q, k = q or side(), k or side()
    pairs = (ctypes.c_int32 * 3)(*split) if split is not None else None
    if bwd:
        return L.svconv_qk_norm_rope_bwd(dtype, d, rot, layout, freq, axes, pairs, eps, ctypes.byref(q), ctypes.byref(k), ws, n, None)
    return L.svconv_qk_norm_rope_fwd(dtype, d, rot, layout, freq, axes, pairs, eps, ctypes.byref(q), ctypes.byref(k), None)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("bad,code", [
    (dict(dtype=sv.E4M3), UNSUP), (dict(d=4), UNSUP), (dict(d=264), UNSUP), (dict(d=60), UNSUP), (dict(rot=24, split=(12,)), UNSUP),
    (dict(rot=80, split=(40,)), UNSUP), (dict(layout=2), UNSUP), (dict(axes=0), SIZE), (dict(axes=4), SIZE), (dict(eps=-1.0), SIZE),
    (dict(eps=math.nan), SIZE), (dict(split=(15,)), SIZE), (dict(axes=2, split=(20, -4)), SIZE), (dict(split=None), NULL),
    (dict(freq=None), NULL), (dict(q=side(n=-1)), SIZE), (dict(k=side(H=0)), SIZE), (dict(q=side(x=None)), NULL),
    (dict(k=side(pos=None)), NULL), (dict(q=side(x_row=252)), ALIGN), (dict(q=side(x_row=128)), ALIGN), (dict(k=side(x=0x10008)), ALIGN),
])
def test_query_key_norm(L, bad, code, backward):
    assert qk(L, bwd=backward, **bad) == code


def test_query_key_norm_outputs_and_workspace(L):
    assert qk(L, q=side(y=None)) == NULL and qk(L, k=side(y=0x10008)) == ALIGN
    assert qk(L, q=side(y=0x10000, x_row=512)) == ALIGN  # in place on strided rows
    assert qk(L, bwd=True, q=side(dy=None)) == NULL and qk(L, bwd=True, k=side(dx=None)) == NULL
    need = L.svconv_qk_norm_rope_bwd_workspace_size(64)
    assert need > 0 and L.svconv_qk_norm_rope_bwd_workspace_size(60) == 0
    assert qk(L, bwd=True, ws=None) == WORKSPACE and qk(L, bwd=True, n=need - 1) == WORKSPACE
    assert qk(L, bwd=True, ws=ODD) == ALIGN


def clip(L, *grads, count=None, max_norm=1.0, norm=A, ws=A, n=1 << 30):
    t = (sv.Grad * max(len(grads), 1))(*grads)
    return L.svconv_clip_grads(t, len(grads) if count is None else count, max_norm, norm, ws, n, None)


def test_clip_grads(L):
    g = lambda src=0x10000, dst=0x10000, numel=10, dtype=sv.F32: sv.Grad(src, dst, numel, dtype)
    assert clip(L, g(numel=-1)) == SIZE and clip(L, g(), count=-1) == SIZE
    assert clip(L, g(dtype=sv.E4M3)) == UNSUP
    assert clip(L, g(src=None)) == NULL and clip(L, g(dst=None)) == NULL and clip(L, g(), norm=None) == NULL
    assert L.svconv_clip_grads(None, 1, 1.0, A, A, 1 << 30, None) == NULL
    assert clip(L, g(src=0x10002)) == ALIGN and clip(L, g(dst=0x10001, dtype=sv.BF16)) == ALIGN and clip(L, g(), ws=ODD) == ALIGN
    assert clip(L, g(), max_norm=-1.0) == SIZE and clip(L, g(), max_norm=math.nan) == SIZE
    assert clip(L, g(), ws=None) == WORKSPACE
    t = (sv.Grad * 1)(g())
    assert clip(L, g(), n=L.svconv_clip_grads_workspace_size(t, 1) - 1) == WORKSPACE


def test_bindings_refuse_what_the_kernels_do_not_take(L):
    import torch
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    off = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):  # CPU tensors
        sv.svconv_cross_attn_fwd(x, x, x, off, off, max_q=4, max_kv=4)
    with pytest.raises(ValueError):
        sv.svconv_qk_norm_rope_fwd(x, x, off, off, torch.zeros(8, dtype=torch.float64))
    with pytest.raises(ValueError):
        sv.svconv_clip_grads([x], 1.0)
    with pytest.raises(ValueError):
        sv.svconv_clip_grads([], 1.0)
