"""What the smaller cache's calls refuse, through the C ABI and the binding (CPU only: nothing is launched)."""
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
ODD = ctypes.c_void_p((1 << 20) + 2)
EIGHT = ctypes.c_void_p((1 << 20) + 8)
INF, NAN = float("inf"), float("nan")


def _run(fn, order, base, kw):
    a = dict(base)
    a.update(kw)
    return fn(*[a[k] for k in order.split()])


def append(L, **kw):
    return _run(L.mla_kv_append_fp4, "c cst k kst w eps q qt qh pos slots cs mp neox T H cache ks np ps qo ot oh kv kvs ws wsb stream",
                dict(c=F, cst=512, k=F, kst=64, w=F, eps=1e-6, q=F, qt=1024, qh=64, pos=F, slots=F, cs=F, mp=64, neox=0, T=4, H=16, cache=F,
                     ks=1.0, np=8, ps=16, qo=F, ot=16 * 576, oh=576, kv=None, kvs=0, ws=F, wsb=256, stream=None), kw)


def decode(L, **kw):
    return _run(L.mla_decode_fp4, "q s cache ks np ps bt mp lens B H scale sinks ns out lse ws wsb stream",
                dict(q=F, s=1, cache=F, ks=1.0, np=8, ps=16, bt=F, mp=4, lens=F, B=2, H=16, scale=0.1, sinks=None, ns=0, out=F, lse=F, ws=F,
                     wsb=1 << 40, stream=None), kw)


def weights(L, **kw):
    return _run(L.mla_key_weights, "q s lse cache fmt ks np ps bt mp lens B H scale decay w st width ws wsb stream",
                dict(q=F, s=1, lse=F, cache=F, fmt=0, ks=1.0, np=8, ps=16, bt=F, mp=4, lens=F, B=2, H=16, scale=0.1, decay=1.0, w=F, st=64,
                     width=64, ws=F, wsb=1 << 40, stream=None), kw)


def select(L, **kw):
    return _run(L.mla_select_keys, "w st width lens keep first recent B K idx count dropped ws wsb stream",
                dict(w=F, st=64, width=64, lens=F, keep=F, first=0, recent=0, B=2, K=8, idx=F, count=F, dropped=F, ws=F, wsb=256, stream=None), kw)


def compact(L, **kw):
    return _run(L.mla_compact_rows, "cache row np ps bt mp idx K count B w st width ws wsb stream",
                dict(cache=F, row=416, np=8, ps=16, bt=F, mp=4, idx=F, K=8, count=F, B=2, w=None, st=0, width=0, ws=F, wsb=256, stream=None), kw)


PAGED = [dict(B=-1), dict(np=-1), dict(mp=-1), dict(ps=0), dict(np=1 << 27), dict(np=1 << 40), dict(mp=1 << 27), dict(bt=None), dict(cache=None),
         dict(cache=EIGHT), dict(bt=ODD)]


@pytest.mark.parametrize("kw", [dict(T=-1), dict(H=-1), dict(mp=0), dict(ps=0), dict(np=-1), dict(np=1 << 27), dict(neox=2), dict(ks=0.0),
                                dict(ks=-1.0), dict(ks=INF), dict(ks=NAN), dict(ks=2.0 ** -101), dict(ks=2.0 ** 101), dict(eps=-1.0), dict(c=None), dict(k=None),
                                dict(pos=None), dict(slots=None), dict(cs=None), dict(cache=None), dict(q=None), dict(qo=None), dict(c=ODD), dict(k=ODD),
                                dict(w=ODD), dict(q=ODD), dict(qo=ODD), dict(cache=ODD), dict(kv=ODD, kvs=576), dict(cst=-8), dict(cst=516), dict(kst=68),
                                dict(kv=F, kvs=568), dict(qt=-8), dict(oh=568), dict(T=1 << 30, H=128), dict(pos=ODD)])
def test_append_refuses(L, kw):
    assert append(L, **kw) == 1 and b"mla_kv_append_fp4" in L.mla_last_error_string()


@pytest.mark.parametrize("kw", PAGED + [dict(s=0), dict(H=0), dict(ns=-1), dict(ns=65536), dict(B=1 << 13, s=1 << 12), dict(scale=NAN), dict(scale=INF),
                                        dict(ks=0.0), dict(ks=-1.0), dict(ks=NAN), dict(ks=2.0 ** -101), dict(ks=2.0 ** 101), dict(q=None), dict(lens=None),
                                        dict(out=None), dict(q=EIGHT), dict(out=EIGHT), dict(lens=ODD), dict(lse=ODD), dict(sinks=ODD), dict(ws=EIGHT)])
def test_decode_refuses(L, kw):
    assert decode(L, **kw) == 1 and b"mla_decode_fp4" in L.mla_last_error_string()


@pytest.mark.parametrize("kw", PAGED + [dict(fmt=-1), dict(fmt=3), dict(s=0), dict(H=0), dict(s=1 << 14, H=128), dict(scale=NAN), dict(ks=0.0), dict(ks=INF),
                                        dict(decay=-0.5), dict(decay=NAN), dict(decay=INF), dict(width=-1), dict(st=-1), dict(q=None), dict(lse=None),
                                        dict(lens=None), dict(w=None), dict(q=EIGHT), dict(lse=ODD), dict(w=ODD), dict(st=63), dict(B=65536)])
def test_weights_refuses(L, kw):
    assert weights(L, **kw) == 1 and b"mla_key_weights" in L.mla_last_error_string()


@pytest.mark.parametrize("kw", [dict(B=-1), dict(K=-1), dict(width=-1), dict(first=-1), dict(recent=-1), dict(st=-1), dict(K=2 ** 31 - 1), dict(width=2 ** 31 - 1),
                                dict(w=None), dict(lens=None), dict(keep=None), dict(idx=None), dict(count=None), dict(dropped=None), dict(w=ODD), dict(lens=ODD),
                                dict(keep=ODD), dict(idx=ODD), dict(count=ODD), dict(dropped=ODD)])
def test_select_refuses(L, kw):
    assert select(L, **kw) == 1 and b"mla_select_keys" in L.mla_last_error_string()


@pytest.mark.parametrize("kw", PAGED + [dict(row=0), dict(row=8), dict(row=418), dict(row=65552), dict(K=-1), dict(width=-1), dict(st=-1), dict(idx=None),
                                        dict(count=None), dict(idx=ODD), dict(count=ODD), dict(w=ODD, st=8, width=8), dict(w=F, st=7, width=8), dict(B=65536)])
def test_compact_refuses(L, kw):
    assert compact(L, **kw) == 1 and b"mla_compact_rows" in L.mla_last_error_string()


def test_more_heads_than_a_tile_are_not_supported(L):
    assert decode(L, H=129) == 2


def test_workspaces_are_required(L):
    for call in (append, decode, weights, select, compact):
        assert call(L, ws=None) == 6 and call(L, wsb=255) == 6
    assert L.mla_decode_fp4_workspace_size(64, 1, 128, 0) >= 256
    assert L.mla_key_weights_workspace_size(64, 1, 128, 32768) == L.mla_select_keys_workspace_size(64) == 256
    assert L.mla_key_weights_workspace_size(64, 2, 128, 32768) >= 256 + 64 * 32768 * 4
    assert weights(L, s=9, wsb=4096) == 6
    assert L.mla_compact_rows_workspace_size(64) == L.mla_kv_append_fp4_workspace_size(64) == 256


def test_nothing_to_do_is_ok(L):
    assert append(L, T=0) == 0 and decode(L, B=0) == 0 and weights(L, B=0) == 0 and select(L, B=0) == 0
    assert compact(L, B=0) == 0 and compact(L, K=0) == 0
    assert L.mla_last_error_string() == b""


def test_the_binding_refuses():
    import mla_attention_gb300 as m
    x, f = torch.zeros((2, 512), dtype=torch.bfloat16), torch.zeros((2, 8))
    i = torch.zeros(2, dtype=torch.int32)
    q, c = torch.zeros((2, 4, 576), dtype=torch.bfloat16), torch.zeros((4, 16, 416), dtype=torch.uint8)
    for call in (lambda: m.mla_kv_append_fp4(x, x[:, :64], i, i, None, c), lambda: m.mla_decode_fp4(q, c, 1.0, i[None], i, 0.1),
                 lambda: m.mla_key_weights(q, f, c, i[None], i, 0.1, f), lambda: m.mla_select_keys(f, i, i, 4),
                 lambda: m.mla_compact_rows(c, i[:, None], i[:, None], i)):
        with pytest.raises(m.MLAError) as e:
            call()
        assert e.value.status == 1 and "CUDA" in str(e.value)
    for call in (lambda: m.mla_decode_fp4(None, c, 1.0, i[None], i, 0.1), lambda: m.mla_key_weights(3, f, c, i[None], i, 0.1, f),
                 lambda: m.mla_select_keys(None, i, i, 4), lambda: m.mla_compact_rows(c, i, None, i)):
        with pytest.raises(m.MLAError):
            call()
