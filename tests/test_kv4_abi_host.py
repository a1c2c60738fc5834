"""Argument checks of the key/value cache's entry points: every call here is
rejected (or has nothing to do) before the library makes a CUDA call, so no
GPU is needed.  Pointers are fake and never dereferenced."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def api():
    from top_selection_dsa_gb300 import build
    build.build()
    from top_selection_dsa_gb300 import api as _api
    return _api


A = ctypes.c_void_p(0x10000)
M8 = ctypes.c_void_p(0x10008)      # 8- but not 16-byte aligned
M2 = ctypes.c_void_p(0x10002)
NUL = None
BIG = 1 << 40


def insert(api, k=A, ks=1024, v=A, vs=1024, slots=A, T=4, hkv=8, D=128, cache=A, sc=A, nb=4,
           bs=64):
    return api.lib.dsa_kv4_insert(k, ks, v, vs, slots, T, hkv, D, cache, sc, nb, bs, NUL)


def test_insert_refusals(api):
    E, U = api.DSA_ERR_INVALID_ARG, api.DSA_ERR_UNSUPPORTED
    for bad in (dict(k=NUL), dict(v=NUL), dict(slots=NUL), dict(cache=NUL), dict(sc=NUL),
                dict(T=-1), dict(hkv=0), dict(nb=0), dict(bs=0), dict(k=M8), dict(v=M8),
                dict(cache=M8), dict(sc=M8), dict(slots=M2), dict(ks=1020), dict(vs=1016),
                dict(ks=-1024), dict(D=0)):
        assert insert(api, **bad) == E, bad
    for bad in (dict(D=96), dict(D=256), dict(bs=4), dict(bs=48), dict(bs=256),
                dict(nb=1 << 30, bs=128)):
        assert insert(api, **bad) == U, bad
    assert insert(api, T=0) == api.DSA_OK


def gather(api, cache=A, sc=A, nb=4, bs=64, slots=A, T=4, hkv=8, D=128, k=A, v=A):
    return api.lib.dsa_kv4_gather(cache, sc, nb, bs, slots, T, hkv, D, k, v, NUL)


def test_gather_refusals(api):
    E, U = api.DSA_ERR_INVALID_ARG, api.DSA_ERR_UNSUPPORTED
    for bad in (dict(cache=NUL), dict(sc=NUL), dict(slots=NUL), dict(k=NUL), dict(v=NUL),
                dict(T=-1), dict(k=M8), dict(v=M8), dict(slots=M2)):
        assert gather(api, **bad) == E, bad
    assert gather(api, D=32) == U and gather(api, bs=24) == U
    assert gather(api, T=0) == api.DSA_OK


def attend(api, sel=None, q=A, cache=A, sc=A, nb=100, bt=A, mb=4, cl=A, B=2, nn=1, bs=64, Hq=64,
           Hkv=8, D=128, scale=0.1, out=A, lse=A, sw=NUL, kw=NUL, ldw=0, ws=A, wsb=BIG, k=16,
           topk=A):
    if sel is None:
        return api.lib.dsa_kv4_attention(q, cache, sc, nb, bt, mb, cl, B, nn, bs, Hq, Hkv, D,
                                         scale, out, lse, kw, ldw, ws, wsb, NUL)
    return api.lib.dsa_kv4_attention_topk(q, cache, sc, nb, bt, mb, cl, topk, k, B, nn, bs, Hq,
                                          Hkv, D, scale, out, lse, sw, kw, ldw, ws, wsb, NUL)


@pytest.mark.parametrize("sel", [None, True])
def test_attention_refusals(api, sel):
    E, U = api.DSA_ERR_INVALID_ARG, api.DSA_ERR_UNSUPPORTED
    for bad in (dict(q=NUL), dict(cache=NUL), dict(sc=NUL), dict(bt=NUL), dict(cl=NUL),
                dict(out=NUL), dict(B=-1), dict(nn=0), dict(mb=0), dict(nb=0), dict(Hq=0),
                dict(Hkv=0), dict(Hq=63), dict(q=M8), dict(out=M2), dict(lse=M2), dict(bt=M2),
                dict(cl=M2), dict(scale=float("inf")), dict(scale=float("nan")),
                dict(kw=A, ldw=255), dict(kw=M2, ldw=256),
                dict(kw=A, ldw=256, wsb=16), dict(kw=A, ldw=256, ws=NUL),
                dict(kw=A, ldw=256, ws=M8)):
        assert attend(api, sel, **bad) == E, bad
    for bad in (dict(D=96), dict(bs=4), dict(bs=100), dict(mb=1 << 24), dict(B=70000),
                dict(nb=1 << 24, bs=128, Hkv=64)):
        assert attend(api, sel, **bad) == U, bad
    assert attend(api, sel, B=0) == api.DSA_OK


def test_attention_topk_refusals(api):
    E = api.DSA_ERR_INVALID_ARG
    for bad in (dict(topk=NUL), dict(topk=M2), dict(k=0), dict(k=-3), dict(sw=M2),
                dict(sw=A, wsb=16)):
        assert attend(api, True, **bad) == E, bad


def test_attention_workspace(api):
    f = api.lib.dsa_kv4_attention_workspace_bytes
    bad = ctypes.c_size_t(-1).value
    for args in ((-1, 1, 8, 8, 128, 64, 0, 0), (1, 0, 8, 8, 128, 64, 0, 0),
                 (1, 1, 9, 8, 128, 64, 0, 0), (1, 1, 8, 0, 128, 64, 0, 0),
                 (1, 1, 8, 8, 0, 64, 0, 0), (1, 1, 8, 8, 128, -1, 0, 0)):
        assert f(*args) == bad, args
    assert f(0, 1, 8, 8, 128, 64, 0, 0) == 0
    # one chunk: nothing but the weights' logits (8 rows of 256 columns and 8
    # heads, fp32) and each row's lse
    assert f(1, 1, 64, 8, 128, 256, 0, 0) == 0
    assert f(1, 1, 64, 8, 128, 256, 0, 1) >= 8 * 8 * 256 * 4 + 8 * 8 * 4
    with pytest.raises(ValueError):
        api.kv4_attention_workspace_bytes(1, 1, 9, 8, 128, 64)


def select(api, kw=A, ldw=512, cl=A, B=2, mc=512, budget=64, sink=4, recent=8, keep=A, nl=A, ws=A,
           wsb=BIG):
    return api.lib.dsa_kv_evict_select(kw, ldw, cl, B, mc, budget, sink, recent, keep, nl, ws, wsb,
                                       NUL)


def test_evict_select_refusals(api):
    E, U = api.DSA_ERR_INVALID_ARG, api.DSA_ERR_UNSUPPORTED
    for bad in (dict(kw=NUL), dict(cl=NUL), dict(keep=NUL), dict(nl=NUL), dict(B=-1), dict(mc=0),
                dict(ldw=511), dict(budget=0), dict(sink=-1), dict(recent=-1), dict(sink=60),
                dict(kw=M2), dict(cl=M2), dict(keep=M2), dict(nl=M2), dict(ws=NUL), dict(ws=M8),
                dict(wsb=8)):
        assert select(api, **bad) == E, bad
    assert select(api, mc=1 << 30, ldw=1 << 30) == U
    assert select(api, B=70000) == U
    assert select(api, B=0) == api.DSA_OK
    w = api.lib.dsa_kv_evict_workspace_bytes
    bad = ctypes.c_size_t(-1).value
    assert w(-1, 10, 4) == bad and w(1, -1, 4) == bad and w(1, 10, 0) == bad
    assert w(2, 512, 64) >= 2 * 4 * 2 + 2 * 64 * 4
    with pytest.raises(ValueError):
        api.kv_evict_workspace_bytes(1, 10, 0)


def compact(api, base=0x10000, planes=8, row=128, n=1, nb=100, bs=64, bt=A, mb=4, nt=A, nmb=4,
            cl=A, keep=A, nl=A, B=2, budget=64, kw=NUL, kwo=NUL, ldw=0, caches=True):
    arr = (api.PagedRows * max(n, 1))(*[api.PagedRows(base, planes, row)] * max(n, 1))
    return api.lib.dsa_kv_compact(arr if caches else None, n, nb, bs, bt, mb, nt, nmb, cl, keep,
                                  nl, B, budget, kw, kwo, ldw, NUL)


def test_compact_refusals(api):
    E, U = api.DSA_ERR_INVALID_ARG, api.DSA_ERR_UNSUPPORTED
    for bad in (dict(caches=False), dict(base=0), dict(base=0x10004), dict(planes=0), dict(row=0),
                dict(row=6), dict(n=-1), dict(nb=0), dict(bs=0), dict(bt=NUL), dict(mb=0),
                dict(nmb=0), dict(cl=NUL), dict(keep=NUL), dict(nl=NUL), dict(B=-1),
                dict(budget=0), dict(kw=A), dict(kwo=A), dict(kw=A, kwo=A, ldw=255),
                dict(kw=M2, kwo=A, ldw=256), dict(keep=M2), dict(bt=M2), dict(nt=M2)):
        assert compact(api, **bad) == E, bad
    for bad in (dict(n=9), dict(bs=48), dict(B=70000), dict(mb=1 << 25), dict(nmb=1 << 25)):
        assert compact(api, **bad) == U, bad
    assert compact(api, B=0) == api.DSA_OK


def test_python_binding_refuses_host_tensors_and_wrong_shapes(api):
    c = torch.zeros(2, 1, 8, 64, dtype=torch.uint8)
    s = torch.zeros(2, 1, 8, 4, dtype=torch.uint8)
    with pytest.raises(ValueError):
        api.kv4_gather(c, s, torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError):
        api.kv4_attention_topk(c, c, s, c, c, None, next_n=1)
    with pytest.raises(ValueError):
        api.kv_evict_select(torch.zeros(1, 8), torch.zeros(1, dtype=torch.int32), 4)
