"""Norm, rotation and append on the GPU against their definitions in 64 bits
(dsa_qk_norm_rope, dsa_kv_append)."""
import math

import pytest
import torch

import kv16_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from top_selection_dsa_gb300 import api as _api
    assert _api.last_device_error() == _api.DSA_OK
    yield _api
    assert _api.last_device_error() == _api.DSA_OK


def rows(seed, T, H, D, extra=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H + extra, D, generator=g, device="cuda")
    x = (x * torch.exp2(2 * torch.randn(T, H + extra, 1, generator=g, device="cuda"))).bfloat16()
    return x[:, :H]


def weights(seed, D):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(D, generator=g, device="cuda")


def close(got, want, tol):
    fine = torch.isfinite(want)
    got = got.double()
    assert torch.equal(torch.isfinite(got), fine)
    worst = ((got - want).abs() / tol)[fine]
    assert worst.numel() == 0 or worst.max().item() <= 1.0, worst.max().item()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,R,norm", [
    (1, 64, 8, 128, 128, True), (1, 1, 0, 64, 16, False), (7, 3, 1, 128, 64, True),
    (33, 64, 1, 128, 64, False), (500, 2, 2, 64, 64, True), (129, 5, 5, 64, 32, False),
    (1000, 1, 1, 128, 112, True), (257, 40, 8, 128, 16, True), (5, 130, 17, 64, 48, True),
])
def test_norm_rope(api, T, Hq, Hk, D, R, norm, interleaved):
    q = rows(T, T, Hq, D, extra=2)
    k = rows(T + 1, T, Hk, D, extra=1) if Hk else None
    pos = torch.randint(-5, 4000, (T,), generator=torch.Generator().manual_seed(T)).int().cuda()
    freq, m = api.rope_frequencies(R, 10000.0)
    qw, kw = (weights(1, D), weights(2, D)) if norm else (None, None)
    if not Hk:
        kw = None
    a, b = api.qk_norm_rope(q, k, pos, api.rope_turns(freq), q_weight=qw, k_weight=kw, eps=1e-5,
                            interleaved=interleaved, rope_scale=m)
    close(a, *ref.norm_rope(q, pos, freq, qw, 1e-5, interleaved, m))
    if Hk:
        close(b, *ref.norm_rope(k, pos, freq, kw, 1e-5, interleaved, m))
    else:
        assert b is None


@pytest.mark.parametrize("opts", [dict(scaling="linear", factor=8.0),
                                  dict(scaling="yarn", factor=40.0, original_context=4096),
                                  dict(base=1e6)])
def test_far_positions(api, opts):
    """The angle is reduced exactly: far positions are as good as near ones."""
    D = R = 128
    pos = torch.tensor([0, 1, 4095, 65537, 999999, 16777217, 2 ** 31 - 1, -2 ** 31]).int().cuda()
    freq, m = api.rope_frequencies(R, **{"base": 10000.0, **opts})
    turns = api.rope_turns(freq)
    q = rows(5, 8, 4, D)
    got, _ = api.qk_norm_rope(q, None, pos, turns, rope_scale=m)
    # angles as the table's whole numbers give them, in exact arithmetic
    angle = [[2 * math.pi * ((int(p) * int(t)) % 2 ** 64) / 2 ** 64 for t in turns.tolist()]
             for p in pos.tolist()]
    t = torch.tensor(angle, dtype=torch.float64, device="cuda")[:, None]
    x = q.double()
    a, b = x[..., :64], x[..., 64:]
    want = m * torch.cat([a * t.cos() - b * t.sin(), a * t.sin() + b * t.cos()], -1)
    size = m * torch.cat([a.abs() + b.abs()] * 2, -1)
    close(got, want, ref.BF16 * want.abs() + (34 * ref.F32 + 2 * math.pi * 2.0 ** -31) * size)


def test_only_norm_and_in_place(api):
    q = rows(3, 50, 6, 64).contiguous()
    w = weights(4, 64)
    want, tol = ref.norm_rope(q, None, None, w, 1e-6)
    a, _ = api.qk_norm_rope(q, None, None, None, q_weight=w)
    close(a, want, tol)
    api.qk_norm_rope(q, None, None, None, q_weight=w, q_out=q)
    assert torch.equal(q, a)
    pos = torch.arange(50, device="cuda", dtype=torch.int32)
    turns = api.rope_turns(api.rope_frequencies(64)[0])
    b, _ = api.qk_norm_rope(q, None, pos, turns)
    api.qk_norm_rope(q, None, pos, turns, q_out=q)
    assert torch.equal(q, b)


def test_rows_that_are_zero_or_not_numbers(api):
    q = rows(6, 4, 3, 128)
    q[0, 0] = 0
    q[1, 1, 100] = math.inf
    q[2, 2, 3] = math.nan
    pos = torch.arange(4, device="cuda", dtype=torch.int32)
    turns = api.rope_turns(api.rope_frequencies(64)[0])
    a, _ = api.qk_norm_rope(q, None, pos, turns)
    assert not a[0, 0].any()
    # element 100 is not rotated: it alone is infinite, and 3 turns with 35
    assert a[1, 1, 100] == math.inf and torch.isfinite(a[1, 1]).sum() == 127
    assert a[2, 2].isnan().nonzero().flatten().tolist() == [3, 35]
    a, _ = api.qk_norm_rope(q, None, pos, turns, q_weight=weights(1, 128))
    assert not a[0, 0].any() and a[2, 2].isnan().all()
    assert torch.isfinite(a[3]).all() and torch.isfinite(a[1, 0]).all()


@pytest.mark.parametrize("queries", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,R,block", [(1, 64, 8, 128, 128, 64), (77, 8, 2, 64, 32, 8),
                                                (400, 12, 3, 128, 64, 128), (3, 1, 1, 64, 0, 16)])
def test_append(api, T, Hq, Hkv, D, R, block, queries):
    k, v = rows(1, T, Hkv, D, extra=1), rows(2, T, Hkv, D, extra=2)
    q = rows(3, T, Hq, D) if queries else None
    nblk = -(-T // block) + 3
    g = torch.Generator().manual_seed(T)
    slots = torch.randperm(nblk * block, generator=g)[:T].cuda()
    if T > 2:
        slots[1] = -1
    kc, vc = api.kv_cache(nblk, Hkv, block, D)
    kc.fill_(3.0)
    vc.fill_(4.0)
    kw = weights(5, D)
    qw = weights(6, D) if queries else None
    pos = torch.arange(T, device="cuda", dtype=torch.int32) + 1000
    freq, m = api.rope_frequencies(R, 5e5) if R else (None, 1.0)
    kc2, vc2, qo = api.kv_append(k, v, slots, kc, vc, positions=pos if R else None,
                                 turns=api.rope_turns(freq) if R else None, k_weight=kw, eps=1e-6,
                                 q=q, q_weight=qw)
    assert kc2 is kc and vc2 is vc and (qo is None) == (not queries)
    ok = slots >= 0
    pg, at = slots[ok] // block, slots[ok] % block
    want, tol = ref.norm_rope(k, pos, freq, kw)
    close(kc[pg, :, at], want[ok], tol[ok])
    assert torch.equal(vc[pg, :, at], v[ok])
    rest = torch.ones(nblk, block, dtype=torch.bool, device="cuda")
    rest[pg, at] = False
    assert (kc.transpose(1, 2)[rest] == 3).all() and (vc.transpose(1, 2)[rest] == 4).all()
    if queries:
        close(qo, *ref.norm_rope(q, pos, freq, qw))
        # the same as the call without a cache, bit for bit
        same, _ = api.qk_norm_rope(q, None, pos if R else None,
                                   api.rope_turns(freq) if R else None, q_weight=qw)
        assert torch.equal(same, qo)


def test_slot_past_the_cache_is_recorded(api):
    k, v = rows(1, 3, 2, 64), rows(2, 3, 2, 64)
    kc, vc = api.kv_cache(2, 2, 8, 64)
    api.kv_append(k, v, torch.tensor([16, 15, 1 << 40], device="cuda"), kc, vc)
    assert api.last_device_error() == api.DSA_ERR_INVALID_ARG
    assert torch.equal(kc[1, :, 7], k[1]) and torch.equal(vc[1, :, 7], v[1])
    kc[1, :, 7] = 0
    assert not kc.any()


def test_graph(api):
    k, v, q = rows(1, 5, 2, 128), rows(2, 5, 2, 128), rows(3, 5, 8, 128)
    kc, vc = api.kv_cache(2, 2, 8, 128)
    slots = torch.arange(5, device="cuda")
    pos = torch.arange(5, device="cuda", dtype=torch.int32)
    turns = api.rope_turns(api.rope_frequencies(128)[0])
    _, _, qo = api.kv_append(k, v, slots, kc, vc, positions=pos, turns=turns, q=q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.kv_append(k, v, slots, kc, vc, positions=pos, turns=turns, q=q, q_out=qo)
    pos += 100
    slots += 7
    graph.replay()
    freq, _ = api.rope_frequencies(128)
    close(qo, *ref.norm_rope(q, pos, freq))
    want, tol = ref.norm_rope(k, pos, freq)
    close(kc[slots // 8, :, slots % 8], want, tol)
