"""Argument checks of the 16-bit cache's entry points: every call here is
rejected (or has nothing to do) before the library makes a CUDA call, so no
GPU is needed.  Pointers are fake and never dereferenced."""
import ctypes
import math

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
M4 = ctypes.c_void_p(0x10004)
M2 = ctypes.c_void_p(0x10002)
NUL = None
BIG = 1 << 40
INF, NAN = math.inf, math.nan


def rope(api, q=A, qs=1024, Hq=8, k=A, ks=256, Hk=2, T=4, D=128, pos=A, turns=A, R=128, il=0,
         m=1.0, qw=A, kw=A, eps=1e-6, qo=A, ko=A):
    return api.lib.dsa_qk_norm_rope(q, qs, Hq, k, ks, Hk, T, D, pos, turns, R, il, m, qw, kw, eps,
                                    qo, ko, NUL)


def test_norm_rope_refusals(api):
    E, U = api.DSA_ERR_INVALID_ARG, api.DSA_ERR_UNSUPPORTED
    for bad in (dict(q=NUL), dict(qo=NUL), dict(ko=NUL), dict(k=NUL), dict(k=NUL, ko=NUL),
                dict(k=NUL, Hk=0), dict(T=-1), dict(Hq=0), dict(Hk=0), dict(D=0), dict(q=M8),
                dict(k=M8), dict(qo=M8), dict(ko=M8), dict(qs=1020), dict(qs=1016), dict(ks=248),
                dict(qs=-1024), dict(R=-16), dict(R=144), dict(R=63), dict(pos=NUL),
                dict(turns=NUL), dict(pos=M2), dict(turns=M4), dict(qw=M2), dict(kw=M2),
                dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(m=INF), dict(m=NAN)):
        assert rope(api, **bad) == E, bad
    for bad in (dict(D=96), dict(D=256), dict(R=8), dict(R=120), dict(Hq=5000, qs=5000 * 128),
                dict(T=1 << 30)):
        assert rope(api, **bad) == U, bad
    assert rope(api, T=0) == api.DSA_OK
    assert rope(api, T=0, k=NUL, ko=NUL, Hk=0, kw=NUL) == api.DSA_OK
    assert rope(api, T=0, R=0, pos=NUL, turns=NUL, qw=NUL, kw=NUL, eps=NAN) == api.DSA_OK


def append(api, k=A, ks=256, v=A, vs=256, slots=A, T=4, hkv=2, D=128, pos=A, turns=A, R=128, il=0,
           m=1.0, kw=A, eps=1e-6, kc=A, vc=A, nb=4, bs=64, q=A, qs=1024, Hq=8, qw=A, qo=A):
    return api.lib.dsa_kv_append(k, ks, v, vs, slots, T, hkv, D, pos, turns, R, il, m, kw, eps, kc,
                                 vc, nb, bs, q, qs, Hq, qw, qo, NUL)


def test_append_refusals(api):
    E, U = api.DSA_ERR_INVALID_ARG, api.DSA_ERR_UNSUPPORTED
    for bad in (dict(k=NUL), dict(v=NUL), dict(slots=NUL), dict(kc=NUL), dict(vc=NUL), dict(T=-1),
                dict(hkv=0), dict(D=0), dict(nb=0), dict(bs=0), dict(k=M8), dict(v=M8),
                dict(kc=M8), dict(vc=M8), dict(slots=M4), dict(ks=252), dict(vs=248),
                dict(q=NUL), dict(q=NUL, qo=NUL), dict(qo=NUL), dict(Hq=0), dict(q=M8),
                dict(qo=M8), dict(qs=1000), dict(pos=NUL), dict(turns=NUL), dict(R=130),
                dict(eps=-1.0), dict(m=INF)):
        assert append(api, **bad) == E, bad
    for bad in (dict(D=96), dict(bs=4), dict(bs=48), dict(bs=256), dict(nb=1 << 25, bs=64),
                dict(R=24), dict(T=1 << 30)):
        assert append(api, **bad) == U, bad
    assert append(api, T=0) == api.DSA_OK
    assert append(api, T=0, q=NUL, qo=NUL, qw=NUL, Hq=0) == api.DSA_OK


def attend(api, q=A, qs=1024, kc=A, vc=A, nb=100, bt=A, mb=4, cl=A, st=A, T=4, B=2, bs=64, Hq=8,
           Hkv=2, D=128, scale=0.1, window=0, sink=0, out=A, lse=A, ws=A, wsb=BIG):
    return api.lib.dsa_kv_attention(q, qs, kc, vc, nb, bt, mb, cl, st, T, B, bs, Hq, Hkv, D, scale,
                                    window, sink, out, lse, ws, wsb, NUL)


def test_attention_refusals(api):
    E, U = api.DSA_ERR_INVALID_ARG, api.DSA_ERR_UNSUPPORTED
    for bad in (dict(q=NUL), dict(kc=NUL), dict(vc=NUL), dict(bt=NUL), dict(cl=NUL), dict(st=NUL),
                dict(out=NUL), dict(T=-1), dict(B=-1), dict(mb=0), dict(nb=0), dict(bs=0),
                dict(Hq=0), dict(Hkv=0), dict(Hq=7), dict(D=0), dict(q=M8), dict(kc=M8),
                dict(vc=M8), dict(out=M8), dict(lse=M2), dict(bt=M2), dict(cl=M2), dict(st=M2),
                dict(qs=1020), dict(qs=512), dict(window=-1), dict(sink=-1), dict(scale=0.0),
                dict(scale=-0.1), dict(scale=INF), dict(scale=NAN), dict(scale=1e30),
                dict(ws=NUL), dict(ws=M8), dict(wsb=1000)):
        assert attend(api, **bad) == E, bad
    for bad in (dict(D=96), dict(bs=4), dict(bs=100), dict(mb=1 << 24), dict(B=2049),
                dict(T=1 << 30), dict(Hq=129, Hkv=1, qs=129 * 128), dict(nb=1 << 25, bs=64),
                dict(T=1 << 28, mb=1 << 23)):
        assert attend(api, **bad) == U, bad
    assert attend(api, B=0) == api.DSA_OK and attend(api, T=0) == api.DSA_OK
    wb = api.lib.dsa_kv_attention_workspace_bytes
    none = ctypes.c_size_t(-1).value
    assert all(wb(*a) == none for a in ((-1, 8, 2, 128), (4, 0, 2, 128), (4, 8, 3, 128),
                                        (4, 8, 2, 96), (4, 129, 1, 64), (4, 8, 0, 64)))
    # rows of one tile, and of two, where a request can have more than one
    assert wb(1, 8, 1, 128) < wb(17, 8, 1, 128) == wb(100000, 8, 1, 128)


def test_frequencies(api):
    freq, m = api.rope_frequencies(64, 10000.0)
    assert m == 1.0 and freq.dtype == torch.float64 and freq.shape == (32,)
    assert freq[0] == 1.0 and abs(freq[16].item() - 1e-2) < 1e-15
    lin, m = api.rope_frequencies(64, 10000.0, scaling="linear", factor=4.0)
    assert m == 1.0 and torch.equal(lin, freq / 4)
    yarn, m = api.rope_frequencies(64, 10000.0, scaling="yarn", factor=40.0, original_context=4096)
    assert abs(m - (0.1 * math.log(40) + 1)) < 1e-15
    turns = 4096 * freq / (2 * math.pi)
    assert torch.equal(yarn[turns > 33], freq[turns > 33])
    slow = turns < 0.7
    assert torch.allclose(yarn[slow], freq[slow] / 40, rtol=1e-12) and slow.any()
    assert ((yarn <= freq) & (yarn >= freq / 40)).all() and (yarn[:-1] >= yarn[1:]).all()
    for bad in (dict(rotary=0), dict(rotary=7), dict(rotary=64, base=1.0),
                dict(rotary=64, factor=0.5, scaling="linear"), dict(rotary=64, factor=2.0),
                dict(rotary=64, scaling="ntk"), dict(rotary=64, scaling="yarn", factor=2.0)):
        with pytest.raises(ValueError):
            api.rope_frequencies(**bad)


def test_turns(api):
    t = api.rope_turns([math.pi, math.pi / 2, 0.0, -math.pi / 2, 1.0], device="cpu")
    assert t.dtype == torch.int64
    u = [int(x) % 2 ** 64 for x in t]
    assert abs(u[0] - 2 ** 63) < 2 ** 12 and abs(u[1] - 2 ** 62) < 2 ** 11 and u[2] == 0
    assert u[3] == 2 ** 64 - u[1]
    # one radian to 64 bits: 2^64 / (2 pi)
    assert u[4] == 2935890503282001226
    for bad in ([math.inf], [math.nan], [2.0 ** 31], [[1.0]]):
        with pytest.raises(ValueError):
            api.rope_turns(bad, device="cpu")


def test_binding_refuses_host_tensors(api):
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    c = torch.zeros(4, 2, 64, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.qk_norm_rope(q, None, i, torch.zeros(64, dtype=torch.int64))
    with pytest.raises(ValueError):
        api.kv_append(q[:, :2], q[:, :2], i.long(), c, c)
    with pytest.raises(ValueError):
        api.kv_attention(q, c, c, torch.zeros(1, 4, dtype=torch.int32), i[:1], i)
