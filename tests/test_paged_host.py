"""Argument checks of the paged calls (no GPU): every refusal comes before
any launch, with the documented status."""

import ctypes

import pytest
import torch

from kv_cache_vector_13_b200 import _lib as L
from kv_cache_vector_13_b200 import api
from test_host_lib import FAKE, quant, view

ODD = FAKE + 2


def plan(R=4, P=16, lens=FAKE, new=FAKE + 64, free=FAKE, cap=8, n_free=FAKE + 128, table=FAKE, ts=8, mp=8, mt=32,
         slots=FAKE, pos=FAKE, cu=FAKE, seq=FAKE + 256, status=FAKE, nout=FAKE + 512):
    return L.lib().tq_page_plan(R, P, lens, new, free, cap, n_free, table, ts, mp, mt, slots, pos, cu, seq, status,
                                nout, None)


@pytest.mark.parametrize("bad", [
    dict(R=-1), dict(P=0), dict(P=-16), dict(mp=-1), dict(mt=-1), dict(cap=-1), dict(ts=-1), dict(ts=7),
    dict(mp=1 << 28, ts=1 << 28), dict(mt=1 << 31), dict(cap=1 << 31), dict(lens=None), dict(new=ODD),
    dict(free=None), dict(n_free=None), dict(table=None), dict(slots=FAKE + 4), dict(pos=None), dict(cu=ODD),
    dict(seq=None), dict(status=None), dict(nout=None), dict(seq=FAKE), dict(nout=FAKE + 128),
])
def test_plan_refusals(bad):
    assert plan(**bad) == L.TQ_EINVAL
    assert L.last_error().startswith("tq_page_plan")


def rope(rot=128, pairing=L.TQ_ROPE_HALF, axes=1, freq=FAKE, axis=None):
    return L.TqRope(rot, pairing, axes, freq, axis)


def append(kq=None, vq=None, r=None, pos=FAKE, ps=0, dt=L.TQ_BF16, T=4, Hq=0, Hkv=2, q=None, qs=(256, 128), k=FAKE,
           ks=(256, 128), v=FAKE, vs=(256, 128), qo=None, kc=None, vc=None, n=8, P=16, slots=FAKE):
    kq, vq = kq or quant(), vq or quant()
    return L.lib().tq_paged_append(
        ctypes.byref(kq), ctypes.byref(vq), None if r is None else ctypes.byref(r), pos, ps, dt, T, Hq, Hkv, q, *qs, k,
        *ks, v, *vs, qo, ctypes.byref(kc or view()), ctypes.byref(vc or view()), n, P, slots, None)


@pytest.mark.parametrize("bad", [
    dict(kq=quant(d=64)), dict(kq=quant(d=100)), dict(dt=9), dict(T=-1), dict(Hkv=-1), dict(n=-1), dict(P=0),
    dict(k=None), dict(k=FAKE + 8), dict(ks=(4, 128)), dict(vs=(256, -8)), dict(v=None), dict(slots=None),
    dict(slots=FAKE + 4), dict(kc=view(norms=None)), dict(vc=view(codes=FAKE + 8)), dict(kc=view(sn=-1)),
    dict(Hq=4, q=FAKE, qo=FAKE + 4096),                      # query rows without a rope
    dict(r=rope(rot=136)), dict(r=rope(rot=24)), dict(r=rope(rot=0)), dict(r=rope(pairing=2)), dict(r=rope(axes=0)),
    dict(r=rope(axes=9)), dict(r=rope(freq=None)), dict(r=rope(axes=3), ps=4), dict(r=rope(axes=3, axis=FAKE), ps=3),
    dict(r=rope(), pos=None), dict(r=rope(), Hq=4, q=FAKE, qo=None), dict(r=rope(), Hq=4, q=FAKE, qo=FAKE),
    dict(r=rope(), Hq=4, q=FAKE + 2, qo=FAKE),
])
def test_append_refusals(bad):
    assert append(**bad) == L.TQ_EINVAL, L.last_error()
    assert L.last_error().startswith("tq_paged_append")


@pytest.mark.parametrize("kq", [quant(bits=3), quant(variant=L.TQ_PROD), quant(rot=L.TQ_ROT_DENSE, rot_matrix=FAKE)])
def test_other_quantizers_are_unsupported(kq):
    assert append(kq=kq) == L.TQ_EUNSUPPORTED
    assert dequant(q=kq) == L.TQ_EUNSUPPORTED
    assert attend(vq=kq) == L.TQ_EUNSUPPORTED


def dequant(q=None, c=None, n=8, P=16, T=4, H=2, slots=FAKE, dt=L.TQ_F32, out=FAKE):
    return L.lib().tq_paged_dequant(ctypes.byref(q or quant()), ctypes.byref(c or view()), n, P, T, H, slots, dt, out,
                                    None)


@pytest.mark.parametrize("bad", [dict(n=-1), dict(n=1 << 31), dict(P=0), dict(T=-1), dict(H=-1), dict(dt=3),
                                 dict(slots=None), dict(out=None), dict(out=FAKE + 8), dict(c=view(norms=None))])
def test_dequant_refusals(bad):
    assert dequant(**bad) == L.TQ_EINVAL


def attend(kq=None, vq=None, q=FAKE, dt=L.TQ_BF16, T=4, Hq=8, Hkv=2, qs=(1024, 128), k=None, v=None, n=8, P=16,
           table=FAKE, ts=8, R=4, mp=8, lens=FAKE, cu=None, mq=1, scale=0.1, causal=1, window=0, out=FAKE + 65536,
           lse=None, ws=FAKE, wsb=1 << 40):
    return L.lib().tq_paged_attention(
        ctypes.byref(kq or quant()), ctypes.byref(vq or quant()), q, dt, T, Hq, Hkv, *qs, ctypes.byref(k or view()),
        ctypes.byref(v or view()), n, P, table, ts, R, mp, lens, cu, mq, scale, causal, window, out, lse, ws, wsb, None)


@pytest.mark.parametrize("bad", [
    dict(kq=quant(d=64)), dict(dt=7), dict(T=-1), dict(Hq=7), dict(Hkv=0), dict(R=-1), dict(T=3), dict(q=None),
    dict(q=FAKE + 2), dict(qs=(1024, 4)), dict(qs=(-8, 128)), dict(n=-1), dict(P=0), dict(table=None), dict(ts=7),
    dict(mp=1 << 28, ts=1 << 28), dict(lens=None), dict(cu=ODD), dict(mq=0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(causal=0, window=4), dict(window=-1), dict(out=None), dict(out=FAKE), dict(lse=ODD),
    dict(k=view(codes=None)), dict(v=view(norms=None)), dict(R=1 << 24, cu=FAKE),
])
def test_attention_refusals(bad):
    assert attend(**bad) == L.TQ_EINVAL, L.last_error()
    assert L.last_error().startswith("tq_paged_attention")


def test_attention_workspace_and_unsupported():
    assert attend(wsb=0) == L.TQ_EWORKSPACE
    assert attend(ws=None) == L.TQ_EWORKSPACE
    assert attend(ws=FAKE + 8) == L.TQ_EWORKSPACE
    assert attend(P=24) == L.TQ_EUNSUPPORTED      # pages of other than a multiple of 16
    assert attend(dt=L.TQ_F32) == L.TQ_EUNSUPPORTED
    f = L.lib().tq_paged_attention_workspace_bytes
    assert f(0, 4, 8, 2, 128) == 0 and f(4, 4, 7, 2, 128) == 0 and f(4, 4, 8, 2, 100) == 0
    # an object for a larger batch serves a smaller one
    for d in (64, 128, 256):
        assert 0 < f(1, 1, 8, 2, d) <= f(4, 64, 8, 2, d) <= f(64, 4096, 8, 2, d)


def test_empty_calls_launch_nothing():
    assert append(T=0, k=None, v=None, slots=None) == L.TQ_OK
    assert append(Hkv=0, k=None, v=None, slots=None) == L.TQ_OK
    assert dequant(T=0, slots=None, out=None) == L.TQ_OK
    assert attend(T=0, R=0, q=None, out=None, lens=None, table=None) == L.TQ_OK


def test_binding_checks():
    f = torch.ones(8)
    assert api.Rope(f).rot_dim == 16
    r = api.Rope(f, sections=(4, 2, 2))
    assert r.n_axes == 3 and r.axis.tolist() == [0, 0, 0, 0, 1, 1, 2, 2]
    assert api.Rope(f, axis=[0, 1] * 4).n_axes == 2
    for bad in (dict(sections=(4, 2)), dict(axis=[0, 1]), dict(pairing="other"), dict(sections=(4, 4), axis=[0] * 8)):
        with pytest.raises(AssertionError):
            api.Rope(f, **bad)
