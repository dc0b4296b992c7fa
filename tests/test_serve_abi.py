"""Refusals of the rotary, 8-bit cache and modified-score entry points: every
argument is checked on the host before anything is launched."""
import ctypes

import pytest
import torch

import block_sparse_bidirectional_select_b200 as sp
import serve_ref as R
from block_sparse_bidirectional_select_b200 import _lib

lib = _lib.load()
GPU = torch.cuda.is_available()
P, MIS, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008), ctypes.c_void_p(0x10001)
INV, UNS, WS = _lib.ERR_INVALID_ARG, _lib.ERR_UNSUPPORTED, _lib.ERR_WORKSPACE
NAN, INF = float("nan"), float("inf")


def rope(X=P, sections=(32,), H=2, L=8, d=64, theta=1e4, Y=P, pos=P, axes=None):
    arr = (ctypes.c_int * max(1, len(sections)))(*sections)
    return lib.sparsed_rope_axes(X, L * d, d, pos, len(sections) if axes is None else axes, ctypes.addressof(arr), H,
                                 L, d, theta, 0, 0, 0, Y, L * d, d, None)


def append(K=P, V=P, N=1, H=1, B=4, C=64, d=64, start=P, count=None, k8=P, v8=P, ks=P, vs=P):
    return lib.sparsed_cache_append(K, 256, 256, 64, V, 256, 256, 64, N, H, B, C, d, start, count, k8, v8, ks, vs,
                                    None)


def attn(Q=P, sn=256, k8=P, v8=P, ks=P, vs=P, N=1, Hq=4, Hkv=2, B=1, C=64, d=64, lengths=P, q_start=None, scale=0.1,
         softcap=0.0, slopes=None, O=P, LSE=P, ws=P, nb=1 << 40):
    return lib.sparsed_cache_attn(Q, sn, 64, 64, k8, v8, ks, vs, N, Hq, Hkv, B, C, d, lengths, q_start, scale,
                                  softcap, slopes, O, LSE, ws, nb, None)


def scored(Q=P, K=P, V=P, sh=512, Hq=4, Hkv=2, Lq=8, Lk=8, d=64, scale=0.1, softcap=0.0, slopes=None, q_start=0,
           ranges=None, O=P, LSE=P, ws=P, nb=1 << 40):
    return lib.sparsed_scored_attn(Q, 512, 64, K, sh, 64, V, 512, 64, Hq, Hkv, Lq, Lk, d, scale, softcap, slopes,
                                   q_start, ranges, O, LSE, ws, nb, None)


@pytest.mark.parametrize("call,kw,status", [
    (rope, dict(X=None), INV), (rope, dict(Y=None), INV), (rope, dict(pos=None), INV), (rope, dict(X=ODD), INV),
    (rope, dict(H=-1), INV), (rope, dict(sections=(-1, 9)), INV), (rope, dict(sections=(0,)), INV),
    (rope, dict(sections=(33,)), INV), (rope, dict(axes=0), INV), (rope, dict(theta=0.5), INV),
    (rope, dict(theta=NAN), INV), (rope, dict(d=60), UNS), (rope, dict(d=520), UNS),
    (rope, dict(sections=(1,) * 9), UNS), (rope, dict(sections=(129,), d=512), UNS),
    (append, dict(K=None), INV), (append, dict(start=None), INV), (append, dict(k8=MIS), INV),
    (append, dict(V=ODD), INV), (append, dict(vs=ODD), INV), (append, dict(C=96), INV), (append, dict(B=65), INV),
    (append, dict(B=-1), INV), (append, dict(d=96), UNS), (append, dict(N=70000), UNS),
    (attn, dict(Q=None), INV), (attn, dict(Q=MIS), INV), (attn, dict(sn=260), INV), (attn, dict(k8=MIS), INV),
    (attn, dict(O=MIS), INV), (attn, dict(lengths=None), INV), (attn, dict(slopes=ODD), INV),
    (attn, dict(Hkv=3), INV), (attn, dict(Hkv=0), INV), (attn, dict(C=32), INV), (attn, dict(scale=-1.0), INV),
    (attn, dict(scale=INF), INV), (attn, dict(softcap=-1.0), INV), (attn, dict(softcap=NAN), INV),
    (attn, dict(d=256), UNS), (attn, dict(N=70000), UNS), (attn, dict(ws=None), WS), (attn, dict(ws=MIS), WS),
    (attn, dict(nb=16), WS),
    (scored, dict(Q=None), INV), (scored, dict(K=None), INV), (scored, dict(V=MIS), INV), (scored, dict(sh=516), INV),
    (scored, dict(Hkv=3), INV), (scored, dict(Lk=-1), INV), (scored, dict(scale=-0.1), INV),
    (scored, dict(softcap=INF), INV), (scored, dict(ranges=ctypes.c_void_p(0x10004)), INV), (scored, dict(O=None), INV),
    (scored, dict(d=80), UNS), (scored, dict(q_start=2 ** 31 - 1), UNS), (scored, dict(ws=None), WS),
    (scored, dict(nb=0), WS),
])
def test_refusals(call, kw, status):
    assert call(**kw) == status


def test_empty_calls_do_nothing():
    for call, kw in ((rope, dict(X=None, Y=None, pos=None, H=0)), (rope, dict(X=None, Y=None, pos=None, L=0)),
                     (append, dict(K=None, V=None, N=0)), (append, dict(B=0)), (attn, dict(Q=None, N=0)),
                     (attn, dict(B=0)), (scored, dict(Hq=0)), (scored, dict(Q=None, Lq=0))):
        assert call(**kw) == _lib.OK


@pytest.mark.skipif(GPU, reason="checks the no-device path")
def test_good_calls_without_a_device():
    for call in (rope, append, attn, scored):
        assert call() == _lib.ERR_NO_DEVICE
    assert lib.sparsed_document_ranges(P, None, 1, 8, P, None) == _lib.ERR_NO_DEVICE


def test_document_ranges_refusals():
    f = lib.sparsed_document_ranges
    assert f(None, None, 1, 8, P, None) == INV
    assert f(P, None, -1, 8, P, None) == INV
    assert f(P, ODD, 1, 8, P, None) == INV
    assert f(P, None, 1, 8, ctypes.c_void_p(0x10004), None) == INV
    assert f(None, None, 1, 0, None, None) == _lib.OK


def test_workspace_sizes():
    for n in (sp.cache_attn_workspace_bytes(1, 8, 2, 1, 128), sp.cache_attn_workspace_bytes(64, 64, 64, 300, 64),
              sp.scored_attn_workspace_bytes(32, 100000), sp.scored_attn_workspace_bytes(1, 1)):
        assert n > 0 and n % 256 == 0
    assert lib.sparsed_cache_attn_workspace_bytes(1, 4, 2, 1, 64, None) == INV
    assert lib.sparsed_scored_attn_workspace_bytes(-1, 4, ctypes.byref(ctypes.c_size_t())) == INV


def test_binding_refusals():
    x = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    pos = torch.zeros(1, 8, dtype=torch.int32)
    with pytest.raises(ValueError):
        sp.rope_axes(x, pos, (32,))                        # not on a GPU
    with pytest.raises(TypeError):
        sp.rope_axes(x.float(), pos, (32,))
    with pytest.raises(ValueError):
        sp.rope_axes(x, pos, (16, 16))                     # positions of one axis
    with pytest.raises(ValueError):
        sp.rope_axes(x.transpose(1, 2), pos, (32,))
    with pytest.raises(ValueError):
        sp.cache_alloc(1, 2, 100, 64, device="cpu")
    c = sp.cache_alloc(1, 2, 128, 64, device="cpu")
    assert c.k8.shape == (1, 2, 128, 64) and c.k_scale.shape == (1, 2, 2)
    start = torch.zeros(1, dtype=torch.int32)
    k = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sp.cache_append(c, k, k, start)                    # not on a GPU
    with pytest.raises(ValueError):
        sp.cache_append(c, k[:, :1], k[:, :1], start)
    with pytest.raises(ValueError):
        sp.cache_append(c, k, k, start.long())
    with pytest.raises(ValueError):
        sp.cache_attn(torch.zeros(1, 3, 1, 64, dtype=torch.bfloat16), c, start)   # 3 query heads on 2
    with pytest.raises(ValueError):
        sp.cache_attn(k, sp.Cache8(c.k8, c.v8, c.k_scale[..., :1], c.v_scale), start)
    with pytest.raises(ValueError):
        sp.scored_attn(x, x[:, :, :32], x[:, :, :32])
    with pytest.raises(ValueError):
        sp.scored_attn(x, x, x, ranges=torch.zeros(7, 2, dtype=torch.int32))


def test_reference_exponents():
    for amax, e in ((448.0, 0), (450.0, 1), (224.0, -1), (1.0, -8), (1.75, -8), (1.7578125, -7), (0.0, -117),
                    (3.3895e38, 119), (1e-40, -117)):
        assert R.exponent(amax) == e
