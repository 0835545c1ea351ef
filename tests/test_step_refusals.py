"""What the serving step's calls refuse, through the C ABI and the binding (CPU only: nothing is launched)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from mla_attention_gb300 import build as b
    b.build()
    from mla_attention_gb300 import _lib
    return _lib.lib()


F = ctypes.c_void_p(1 << 20)
FAR = ctypes.c_void_p(1 << 21)
ODD = ctypes.c_void_p((1 << 20) + 2)
BYTE = ctypes.c_void_p((1 << 20) + 1)


def _run(fn, order, base, kw):
    a = dict(base)
    a.update(kw)
    return fn(*[a[k] for k in order.split()])


def slot_map(L, **kw):
    return _run(L.mla_slot_map, "lens new B bt mp ps np pool st N cu pos slots lo so ws wsb stream",
                dict(lens=F, new=F, B=2, bt=F, mp=4, ps=16, np=8, pool=F, st=F, N=4, cu=F, pos=F, slots=FAR, lo=F, so=F, ws=F, wsb=256,
                     stream=None), kw)


def norm(L, **kw):
    return _run(L.mla_rms_norm, "x xs r rs w eps T D ro ros e4m3 group out os scales stream",
                dict(x=F, xs=512, r=None, rs=0, w=F, eps=1e-6, T=2, D=512, ro=None, ros=0, e4m3=0, group=0, out=F, os=512, scales=None,
                     stream=None), kw)


def append(L, **kw):
    return _run(L.mla_kv_append, "c cst k kst w eps q qt qh pos slots cs mp neox T H cache e4m3 ks np ps qo ot oh kv kvs ws wsb stream",
                dict(c=F, cst=512, k=F, kst=64, w=F, eps=1e-6, q=F, qt=1024, qh=64, pos=F, slots=F, cs=F, mp=64, neox=0, T=4, H=16, cache=F,
                     e4m3=0, ks=1.0, np=8, ps=16, qo=F, ot=16 * 576, oh=576, kv=None, kvs=0, ws=F, wsb=256, stream=None), kw)


def w4(L, **kw):
    return _run(L.mla_bmm_w4, "x xt xh w s f32 group T H N K out ot oh ws wsb stream",
                dict(x=F, xt=256, xh=128, w=F, s=F, f32=0, group=64, T=2, H=2, N=32, K=128, out=F, ot=64, oh=32, ws=F, wsb=256, stream=None), kw)


@pytest.mark.parametrize("kw", [dict(B=-1), dict(N=-1), dict(mp=-1), dict(ps=0), dict(np=-1), dict(np=1 << 27), dict(np=1 << 40), dict(lens=None),
                                dict(new=None), dict(bt=None), dict(pool=None), dict(st=None), dict(cu=None), dict(pos=None), dict(slots=None),
                                dict(slots=F), dict(lo=None), dict(so=None), dict(slots=BYTE), dict(lens=ODD), dict(so=ODD)])
def test_slot_map_refuses(L, kw):
    assert slot_map(L, **kw) == 1 and b"mla_slot_map" in L.mla_last_error_string()


def test_workspaces_are_required(L):
    assert slot_map(L, ws=None) == 6 and slot_map(L, wsb=16) == 6
    assert append(L, ws=None) == 6 and append(L, wsb=255) == 6
    assert w4(L, ws=None) == 6 and w4(L, wsb=255) == 6
    assert L.mla_slot_map_workspace_size(5) == L.mla_kv_append_workspace_size(5) == 256


@pytest.mark.parametrize("kw,status", [(dict(T=-1), 1), (dict(D=0), 1), (dict(D=32769, xs=40000, os=40000), 2), (dict(eps=-1.0), 1),
                                       (dict(eps=float("nan")), 1), (dict(e4m3=2), 1), (dict(e4m3=1), 1), (dict(scales=F), 1), (dict(group=64), 1),
                                       (dict(e4m3=1, scales=F, group=48), 1), (dict(e4m3=1, scales=F, group=128, D=192), 1), (dict(r=F), 1),
                                       (dict(ro=F), 1), (dict(x=None), 1), (dict(w=None), 1), (dict(out=None), 1), (dict(x=BYTE), 1),
                                       (dict(out=BYTE), 1), (dict(e4m3=1, scales=ODD), 1), (dict(xs=-1), 1), (dict(os=511), 1),
                                       (dict(r=F, ro=F, rs=512, ros=500), 1)])
def test_norm_refuses(L, kw, status):
    assert norm(L, **kw) == status and b"mla_rms_norm" in L.mla_last_error_string()


@pytest.mark.parametrize("kw", [dict(T=-1), dict(H=-1), dict(mp=0), dict(ps=0), dict(np=-1), dict(np=1 << 27), dict(neox=2), dict(e4m3=2),
                                dict(e4m3=1, ks=0.0), dict(e4m3=1, ks=-1.0), dict(e4m3=1, ks=float("inf")), dict(eps=-1.0), dict(c=None), dict(k=None),
                                dict(pos=None), dict(slots=None), dict(cs=None), dict(cache=None), dict(q=None), dict(qo=None), dict(c=ODD), dict(k=ODD),
                                dict(w=ODD), dict(q=ODD), dict(qo=ODD), dict(cache=ODD), dict(kv=ODD, kvs=576), dict(cst=-8), dict(cst=516), dict(kst=68),
                                dict(kv=F, kvs=568), dict(kv=F, kvs=580), dict(qt=-8), dict(qh=66), dict(oh=568), dict(ot=16 * 576 - 8), dict(oh=580),
                                dict(T=1 << 30, H=128), dict(pos=ODD), dict(slots=BYTE)])
def test_append_refuses(L, kw):
    assert append(L, **kw) == 1 and b"mla_kv_append" in L.mla_last_error_string()


@pytest.mark.parametrize("kw", [dict(T=-1), dict(H=0), dict(N=0), dict(K=0), dict(group=16), dict(group=48), dict(K=96), dict(f32=2), dict(x=None),
                                dict(w=None), dict(s=None), dict(out=None), dict(x=BYTE), dict(out=BYTE), dict(s=BYTE), dict(s=ODD, f32=1), dict(w=ODD),
                                dict(xt=-1), dict(xh=-1), dict(ot=32), dict(oh=31), dict(H=70000), dict(H=60000, N=60000), dict(T=(1 << 19) + 1),
                                dict(K=(1 << 30) + 64)])
def test_w4_refuses(L, kw):
    assert w4(L, **kw) == 1 and b"mla_bmm_w4" in L.mla_last_error_string()


def test_nothing_to_do_is_ok(L):
    assert norm(L, T=0) == 0 and append(L, T=0) == 0 and w4(L, T=0) == 0
    assert L.mla_last_error_string() == b""


def test_the_binding_refuses_host_tensors():
    import mla_attention_gb300 as m
    x = torch.zeros((2, 512), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: m.mla_rms_norm(x, x[0]), lambda: m.mla_slot_map(i, i, i[None], i, i, 16, 4),
                 lambda: m.mla_kv_append(x, x[:, :64], i, i, None, None), lambda: m.mla_bmm_w4(x[None], None, None)):
        with pytest.raises(m.MLAError) as e:
            call()
        assert e.value.status == 1 and "CUDA" in str(e.value)
