"""The 4-bit cache's attention where sizes, scales and masks are far apart:
long contexts, scales that grow along them, and what rows do not see, against
the formulas in 64 bits (torch, on the GPU).

Tolerances are those of test_kv4_gpu.py's first lines, with B = |scale| max_c
sum_d |q_d||k_d| of a row and dS = (2^-19 + 2^-24) B:
  weights  e^(error of the logits) on the numerator and in the log-sum-exp, ex2
           within 2^-21, fp32 sums: relative 2 dS + 2^-18; then one fp32
           addition a row: 2^-24 of the sum for each.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import kv4_reference as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from top_selection_dsa_gb300 import api as _api
    return _api


@pytest.fixture(autouse=True)
def clean_error_word(api):
    yield
    assert api.last_device_error() == api.DSA_OK


class Cache:
    """Random codes under given scale codes: key_codes, value_codes [L, Hkv,
    D/32] of each request; pages in random order."""

    def __init__(self, lens, nn, Hq, Hkv, D, bs, key_codes, value_codes, q, seed=0, codes=255):
        rng = np.random.default_rng(seed)
        nblk = [max(-(-L // bs), 1) for L in lens]
        total = sum(nblk)
        perm = rng.permutation(total).astype(np.int32)
        table = np.zeros((len(lens), max(nblk)), np.int32)
        self.rec = rng.integers(0, 256, size=(total, Hkv, bs, D), dtype=np.uint8) & codes
        self.sc = np.full((total, Hkv, bs, D // 16), 127, np.uint8)
        self.K, self.V = [], []
        at = 0
        for b, L in enumerate(lens):
            table[b, :nblk[b]] = perm[at:at + nblk[b]]
            at += nblk[b]
            pos = np.arange(L)
            page, row = table[b, pos // bs], pos % bs
            self.sc[page, :, row] = np.concatenate([key_codes[b], value_codes[b]], -1)
            k, v = ref.decode(self.rec[page, :, row], self.sc[page, :, row]) if L else \
                (np.zeros((0, Hkv, D)),) * 2
            self.K.append(torch.from_numpy(k).cuda())
            self.V.append(torch.from_numpy(v).cuda())
        self.lens, self.nn, self.Hq, self.Hkv, self.D, self.bs = lens, nn, Hq, Hkv, D, bs
        self.table = table
        self.q = torch.as_tensor(q).float().bfloat16().cuda().reshape(len(lens) * nn, Hq, D)
        self.args = (self.q, torch.from_numpy(self.rec).cuda(), torch.from_numpy(self.sc).cuda(),
                     torch.from_numpy(table).cuda(),
                     torch.tensor(lens, dtype=torch.int32, device="cuda"))

    def row(self, b, j, scale):
        """Row j of request b in 64 bits: (out [Hq, D], lse [Hq], weights [Hq,
        L], sum p |V| [Hq, D], B [Hq])."""
        L, G = self.lens[b], self.Hq // self.Hkv
        n = max(L - self.nn + j + 1, 0)
        q = self.q[b * self.nn + j].double()
        K = self.K[b][:n].repeat_interleave(G, 1)            # [n, Hq, D]
        V = self.V[b][:n].repeat_interleave(G, 1)
        S = scale * torch.einsum("hd,nhd->hn", q, K)
        B = abs(scale) * torch.einsum("hd,nhd->hn", q.abs(), K.abs()).amax(1)
        lse = torch.logsumexp(S, 1)
        p = torch.exp(S - lse[:, None])
        w = torch.zeros(self.Hq, L, dtype=torch.float64, device="cuda")
        w[:, :n] = p
        return (torch.einsum("hn,nhd->hd", p, V), lse, w,
                torch.einsum("hn,nhd->hd", p, V.abs()), B)


def rel_of(B):
    return 2 * (2.0 ** -19 + 2.0 ** -24) * float(B.max()) + 2.0 ** -18


# --------------------------------------------------------- every key's weight


@pytest.mark.parametrize("rows", [24, 40, 64])
def test_weights_over_many_tiles_of_growing_keys(api, rows):
    """131071 keys whose scales grow by 2^9 along the context: each call's
    weights are those in 64 bits and of the same keys selected, and those of
    every other call to the bit."""
    L, D = 131071, 128
    rng = np.random.default_rng(rows)
    grow = (np.arange(L) * 10 // L)[:, None, None]
    kc = 118 + grow + rng.integers(-1, 2, size=(L, 1, 4))
    vc = rng.integers(125, 129, size=(L, 1, 4))
    scale = 0.02
    c = Cache([L], 1, rows, 1, D, 64, [kc], [vc], rng.standard_normal((rows, D)), seed=rows)
    out, lse, p, A, B = c.row(0, 0, scale)
    want = p.sum(0)
    rel = rel_of(B)
    width = c.table.shape[1] * 64
    first = None
    for _ in range(20):
        acc = torch.zeros(1, width, device="cuda")
        api.kv4_attention(*c.args, next_n=1, softmax_scale=scale, key_weights=acc)
        if first is None:
            first = acc
        assert torch.equal(acc, first)
    got = first[0, :L].double()
    tol = (rel + rows * 2.0 ** -24) * want
    assert ((got - want).abs() <= tol).all(), float(((got - want).abs() / want).max())
    assert (first[0, L:] == 0).all()
    sel = torch.arange(L, dtype=torch.int32, device="cuda")[None]
    sw = torch.empty(1, L, device="cuda")
    api.kv4_attention_topk(*c.args, sel, next_n=1, softmax_scale=scale, sel_weights=sw)
    assert ((sw[0].double() - want).abs() <= tol).all()


# ------------------------------------------------------------------ compaction


@pytest.mark.parametrize("alone", [False, True])
def test_a_new_table_too_short_for_the_kept_rows_is_reported(api, alone):
    """12 rows kept, pages for 8: the first 8 move, with their weights, the rest
    are zeros and the call is reported."""
    bs = 8
    g = torch.arange(4 * bs, dtype=torch.int32, device="cuda").reshape(4, bs).clone()
    before = g.clone()
    keep = torch.arange(2, 14, dtype=torch.int32, device="cuda")[None]
    cl = torch.tensor([16], dtype=torch.int32, device="cuda")
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    fresh = torch.tensor([[3]], dtype=torch.int32, device="cuda")
    n = torch.tensor([12], dtype=torch.int32, device="cuda")
    w = torch.arange(1, 17, dtype=torch.float32, device="cuda")[None].clone()
    out = w if alone else torch.full_like(w, 5.0)
    api.kv_compact([g], keep, cl, table, fresh, new_lens=n, key_weights=w, key_weights_out=out)
    assert api.last_device_error() == api.DSA_ERR_INVALID_ARG
    before[3] = torch.arange(2, 10, dtype=torch.int32)
    assert torch.equal(g, before)
    assert out[0].tolist() == list(range(3, 11)) + [0.0] * 8


def test_more_rows_than_the_table_has_room_for_in_place_are_reported(api):
    bs = 8
    g = torch.arange(4 * bs, dtype=torch.int32, device="cuda").reshape(4, bs).clone()
    before = g.clone()
    keep = torch.arange(20, dtype=torch.int32, device="cuda")[None]
    cl = torch.tensor([16], dtype=torch.int32, device="cuda")
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    n = torch.tensor([20], dtype=torch.int32, device="cuda")
    w = torch.arange(1, 17, dtype=torch.float32, device="cuda")[None].clone()
    w0 = w.clone()
    api.kv_compact([g], keep, cl, table, new_lens=n, key_weights=w)
    assert api.last_device_error() == api.DSA_ERR_INVALID_ARG
    assert torch.equal(g, before) and torch.equal(w, w0)


# ------------------------------------------------------------------ no requests


def test_calls_without_requests_return_what_there_is(api):
    """An empty batch: outputs of no rows, nothing touched."""
    cache, scales = api.kv4_cache(2, 2, 8, 64)
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    lens = torch.empty(0, dtype=torch.int32, device="cuda")
    out, lse = api.kv4_attention(q, cache, scales, table, lens, next_n=2)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    sel = torch.empty(0, 5, dtype=torch.int32, device="cuda")
    acc = torch.empty(0, 24, device="cuda")
    out, lse = api.kv4_attention_topk(q, cache, scales, table, lens, sel, next_n=2,
                                      key_weights=acc)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    keep, n = api.kv_evict_select(acc, lens, 4)
    assert keep.shape == (0, 4) and n.shape == (0,)
    api.kv_compact([cache, scales], keep, lens, table, key_weights=acc)
    assert (cache == 0).all() and (scales == 0).all()


# ------------------------------------------------- what a row does not see


def check_row(c, out, lse, b, j, scale, under=2.0 ** -24):
    """Row j of request b: output within fp16 weights' rounding (2^-11), the
    logits', bf16's (2^-8), and the sums of what fp16 cannot hold, `under` of the
    32-channel block's largest visible value each; its log-sum-exp."""
    want, wlse, w, A, B = c.row(b, j, scale)
    n = max(c.lens[b] - c.nn + j + 1, 0)
    dS = (2.0 ** -19 + 2.0 ** -24) * B
    G = c.Hq // c.Hkv
    top = c.V[b][:n].abs().reshape(n, c.Hkv, c.D // 32, 32).amax((0, 3))
    top = top.repeat_interleave(G, 0).repeat_interleave(32, 1)
    tol = A * (2.0 ** -11 + 2 * dS + 2.0 ** -18)[:, None] + n * under * top + 2.0 ** -8 * want.abs()
    r = b * c.nn + j
    err = (out[r].double() - want).abs()
    assert (err <= tol).all(), (b, j, float((err / tol).max()))
    err = (lse[r].double() - wlse).abs()
    assert (err <= 2 * dS + 2.0 ** -18 + 2.0 ** -22 * wlse.abs()).all(), (b, j, float(err.max()))


@pytest.mark.parametrize("far", [20, 60, 100])
@pytest.mark.parametrize("Hq,nn", [(4, 2), (8, 2), (16, 2), (32, 2), (16, 4), (10, 3)])
def test_finite_keys_of_later_tokens_do_not_reach_a_row(api, Hq, nn, far):
    """The request's new tokens after a row's own have key scales up to 2^far of
    the others': the row stays as exact as without them."""
    lens, D = [200, 129, 3], 128
    rng = np.random.default_rng(far + Hq)
    kc = [rng.integers(126, 129, size=(L, 1, 4)) for L in lens]
    vc = [rng.integers(126, 129, size=(L, 1, 4)) for L in lens]
    for b, L in enumerate(lens):
        for j in range(1, nn):
            if L - nn + j >= 0:
                kc[b][L - nn + j, 0, j % 4] += far * j // (nn - 1)
    c = Cache(lens, nn, Hq, 1, D, 64, kc, vc, rng.standard_normal((len(lens) * nn * Hq, D)),
              seed=far)
    out, lse = api.kv4_attention(*c.args, next_n=nn, softmax_scale=0.05)
    assert torch.isfinite(out.float()).all()
    for b, L in enumerate(lens):
        if L - nn + 1 > 0:
            check_row(c, out, lse, b, 0, 0.05)


@pytest.mark.parametrize("rows", [8, 16, 24, 64])
@pytest.mark.parametrize("step", [1, -1])
def test_key_scales_far_apart_within_a_context(api, rows, step):
    """Keys whose scales rise (or fall) by 2^40 along the context, and by 2^10
    between the blocks of one: the logits are the formula's."""
    L, D = 700, 128
    rng = np.random.default_rng(rows)
    at = np.arange(L)[::step]
    kc = (107 + at * 40 // L)[:, None, None] + rng.integers(-5, 6, size=(L, 1, 4))
    vc = rng.integers(126, 129, size=(L, 1, 4))
    scale = 2.0 ** -17
    c = Cache([L], 1, rows, 1, D, 64, [kc], [vc], rng.standard_normal((rows, D)), seed=rows)
    out, lse = api.kv4_attention(*c.args, next_n=1, softmax_scale=scale)
    check_row(c, out, lse, 0, 0, scale)


@pytest.mark.parametrize("far", [6, 20, 60, 100])
@pytest.mark.parametrize("Hq,nn", [(4, 2), (8, 2), (16, 2), (32, 2), (16, 4), (10, 3), (1, 40)])
def test_finite_values_of_later_tokens_do_not_reach_a_row(api, Hq, nn, far):
    """The new tokens' value scales rise to 2^far of the others': every row is as
    exact as the values that it sees allow, block by block, and so are the keys'
    weights."""
    lens, D = [200, 129, 64, 300, 3], 128
    rng = np.random.default_rng(far + Hq)
    kc = [rng.integers(126, 129, size=(L, 1, 4)) for L in lens]
    vc = [rng.integers(126, 129, size=(L, 1, 4)) for L in lens]
    for b, L in enumerate(lens):
        for j in range(1, nn):
            if L - nn + j >= 0:
                vc[b][L - nn + j, 0, [j % 4, (j + b) % 4]] += far * j // (nn - 1)
    c = Cache(lens, nn, Hq, 1, D, 64, kc, vc, rng.standard_normal((len(lens) * nn * Hq, D)),
              seed=far)
    out, lse = api.kv4_attention(*c.args, next_n=nn, softmax_scale=0.05)
    acc = torch.zeros(len(lens), c.table.shape[1] * 64, device="cuda")
    out2, lse2 = api.kv4_attention(*c.args, next_n=nn, softmax_scale=0.05, key_weights=acc)
    assert torch.equal(out.view(torch.int16), out2.view(torch.int16)) and torch.equal(lse, lse2)
    for b, L in enumerate(lens):
        want, most = torch.zeros(L, dtype=torch.float64, device="cuda"), 0.0
        for j in range(nn):
            if L - nn + j + 1 <= 0:
                assert (out[b * nn + j] == 0).all() and (lse[b * nn + j] == -torch.inf).all()
                continue
            check_row(c, out, lse, b, j, 0.05)
            row = c.row(b, j, 0.05)
            want += row[2].sum(0)
            most = max(most, rel_of(row[4]))
        tol = (most + nn * Hq * 2.0 ** -24) * want
        assert ((acc[b, :L].double() - want).abs() <= tol).all(), b
        assert (acc[b, L:] == 0).all()


@pytest.mark.parametrize("rows", [8, 16, 24, 64])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["blocks", "rise", "fall", "keys"])
def test_value_scales_far_apart(api, rows, D, kind):
    """Value scales 2^+-18 apart between the blocks of a head (each is as exact as
    alone), rising or falling by 2^60 along the context, or 2^+-18 at random."""
    L, G = 700, D // 32
    rng = np.random.default_rng(rows)
    kc = rng.integers(126, 129, size=(L, 1, G))
    vc = rng.integers(126, 129, size=(L, 1, G))
    if kind == "blocks":
        vc += (np.arange(G) * 37 // G - 18)[None, None]
    elif kind == "keys":
        vc += rng.integers(-18, 19, size=(L, 1, G))
    else:
        vc += (np.arange(L)[::1 if kind == "rise" else -1] * 60 // L - 30)[:, None, None]
    c = Cache([L], 1, rows, 1, D, 64, [kc], [vc], rng.standard_normal((rows, D)), seed=rows)
    for call in ("every", "selected"):
        if call == "every":
            out, lse = api.kv4_attention(*c.args, next_n=1, softmax_scale=0.1)
        else:
            sel = torch.randperm(L, dtype=torch.int32, device="cuda")[None]
            out, lse = api.kv4_attention_topk(*c.args, sel, next_n=1, softmax_scale=0.1)
        check_row(c, out, lse, 0, 0, 0.1)


@pytest.mark.parametrize("rows", [4, 16, 24, 64])
@pytest.mark.parametrize("scale", [1e-42, -1e-42])
def test_a_factor_below_the_smallest_number_leaves_masked_columns_out(api, rows, scale):
    """Queries of 2^-30 under a subnormal softmax scale: all logits are zero to
    any precision, and the columns that are not there still have no weight."""
    L, D = 150, 128
    rng = np.random.default_rng(rows)
    kc = rng.integers(126, 129, size=(L, 1, 4))
    vc = rng.integers(126, 129, size=(L, 1, 4))
    q = rng.standard_normal((2 * rows // 2, D)) * 2.0 ** -30
    c = Cache([L], 2, rows // 2, 1, D, 64, [kc], [vc], q, seed=rows)
    out, lse = api.kv4_attention(*c.args, next_n=2, softmax_scale=scale)
    for j in range(2):
        check_row(c, out, lse, 0, j, scale)
    sel = torch.randperm(L - 1, dtype=torch.int32, device="cuda")[None].repeat(2, 1)
    sel[:, 5::7] = -1
    out, lse = api.kv4_attention_topk(*c.args, sel, next_n=2, softmax_scale=scale)
    keep = sel[0][sel[0] >= 0].long()
    want = c.V[0][keep, 0].mean(0)
    top = c.V[0][keep, 0].abs().mean(0)
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * top).all()
    assert ((lse.double() - np.log(len(keep))).abs() <= 2.0 ** -18 + 2.0 ** -20).all()


@pytest.mark.parametrize("rows", [8, 16, 24, 64])
@pytest.mark.parametrize("L", [90, 700, 5000])
def test_the_mean_of_values_whose_sum_is_no_number(api, rows, L):
    """Positive values around 2^123: their weighted sum overflows fp32, their
    mean does not."""
    D = 128
    rng = np.random.default_rng(rows)
    kc = rng.integers(124, 127, size=(L, 1, 4))
    vc = rng.integers(246, 249, size=(L, 1, 4))
    q = rng.standard_normal((rows, D))
    c = Cache([L], 1, rows, 1, D, 64, [kc], [vc], q, seed=rows, codes=0x77)
    out, lse = api.kv4_attention(*c.args, next_n=1, softmax_scale=0.05)
    check_row(c, out, lse, 0, 0, 0.05)
    sel = torch.randperm(L, dtype=torch.int32, device="cuda")[None]
    out, lse = api.kv4_attention_topk(*c.args, sel, next_n=1, softmax_scale=0.05)
    check_row(c, out, lse, 0, 0, 0.05)


@pytest.mark.parametrize("rows", [1, 8, 16, 24, 64])
@pytest.mark.parametrize("what", ["every", "selected"])
def test_many_small_weights_beside_large_ones(api, rows, what):
    """Four keys (one in each warp's first tile) take nearly all the weight and
    have small values; the output is the other 32764 keys', each at 2^-25.2 of
    one's weight.  What fp16 cannot hold of a term, two half steps of 2^-24 in
    units of 2^-5 of the largest weight, is 2^-28 of that and the largest value,
    and the sum of the weights is 4.  300 requests on the same pages, so that a
    CTA has long runs of columns."""
    L, D, B = 32768, 128, 300
    rng = np.random.default_rng(rows)
    kc = np.full((L, 1, 4), 107)
    vc = np.full((L, 1, 4), 127)
    big = [0, 64, 128, 192]
    kc[big], vc[big] = 127, 100
    q = 1 + 2.0 ** -6 * rng.standard_normal((rows, D))
    c = Cache([L], 1, rows, 1, D, 64, [kc], [vc], q, seed=rows, codes=0x77)
    for pos in big:
        c.args[1][int(c.table[0, pos // 64]), 0, pos % 64, :D // 2] = 0x22    # every element 1
        c.K[0][pos] = 1.0
    scale = 25.2 * np.log(2) / 128
    qs, rec, sc, table, lens = c.args
    args = (qs.repeat(B, 1, 1), rec, sc, table.repeat(B, 1), lens.repeat(B))
    if what == "every":
        out, lse = api.kv4_attention(*args, next_n=1, softmax_scale=scale)
    else:
        sel = torch.arange(L, dtype=torch.int32, device="cuda")[None].repeat(B, 1)
        out, lse = api.kv4_attention_topk(*args, sel, next_n=1, softmax_scale=scale)
    for b in (0, 1, 2, 150, 299):
        check_row(c, out[b:b + 1], lse[b:b + 1], 0, 0, scale, under=2.0 ** -30)


# ------------------------------------------------------------------- NaN scales


@pytest.mark.parametrize("Hq,nn", [(8, 1), (16, 1), (24, 1), (64, 1), (12, 2), (32, 2)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", ["value", "key", "last"])
def test_nan_scales_reach_the_rows_that_see_them(api, Hq, nn, D, bad):
    """A value block's NaN scale is its 32 channels' of every row that sees the
    token, a key block's all of the row's; other rows, channels and keys' weights
    are as exact as without."""
    L, G = 400, D // 32
    rng = np.random.default_rng(Hq + D)
    kc = rng.integers(126, 129, size=(L, 1, G))
    vc = rng.integers(126, 129, size=(L, 1, G))
    q = rng.standard_normal((nn * Hq, D))
    block = G - 1
    pos = L - 1 if bad == "last" else 137
    if bad == "value":
        vc[pos, 0, block] = 255
    else:
        kc[pos, 0, block] = 255
        vc[pos, 0, 0] = 255
    c = Cache([L], nn, Hq, 1, D, 16, [kc], [vc], q, seed=Hq)
    acc = torch.zeros(1, L, device="cuda")
    out, lse = api.kv4_attention(*c.args, next_n=nn, softmax_scale=0.05, key_weights=acc)
    c.V[0] = torch.nan_to_num(c.V[0])
    clean, want = [], torch.zeros(L, dtype=torch.float64, device="cuda")
    for j in range(nn):
        if bad == "value":
            lane = torch.zeros(D, dtype=torch.bool, device="cuda")
            lane[32 * block:32 * block + 32] = True
            assert torch.isnan(out[j][:, lane]).all() and torch.isfinite(lse[j]).all()
            o = torch.where(lane, c.row(0, j, 0.05)[0], out[j].double())
            check_row(c, torch.stack([o] * nn), lse, 0, j, 0.05)
            clean.append(j)
        elif bad == "last" and j < nn - 1:
            check_row(c, out, lse, 0, j, 0.05)
            clean.append(j)
        else:
            assert torch.isnan(out[j]).all() and torch.isnan(lse[j]).all()
    if len(clean) == nn:
        rows = [c.row(0, j, 0.05) for j in range(nn)]
        want = sum(r[2].sum(0) for r in rows)
        rel = max(rel_of(r[4]) for r in rows)
        assert ((acc[0].double() - want).abs() <= (rel + nn * Hq * 2.0 ** -24) * want).all()
    else:
        assert torch.isnan(acc[0]).all()
    c.V[0] = torch.nan_to_num(c.V[0])
    sel = torch.randperm(L - nn + 1, dtype=torch.int32, device="cuda")[None].repeat(nn, 1)
    sel = sel[:, :300].contiguous()
    sel = torch.where(sel == pos, torch.full_like(sel, -1), sel)
    out, lse = api.kv4_attention_topk(*c.args, sel, next_n=nn, softmax_scale=0.05)
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()


# --------------------------------------------------------------------- eviction


@pytest.mark.parametrize("B,ctx", [(3, 900), (160, 900), (3, 40000)])
def test_weights_that_are_no_numbers_are_never_chosen(api, B, ctx):
    """On both of the selection's paths: NaN and -inf in the middle, more and
    fewer numbers left than there is room for; sink and recent stay."""
    rng = np.random.default_rng(ctx)
    w = np.exp(rng.standard_normal((B, ctx))).astype(np.float32)
    lens = rng.integers(1, ctx + 1, size=B)
    lens[:3] = ctx, ctx // 2, ctx // 3
    for b in range(B):
        share = (0.1, 0.95, 1.0)[b % 3]
        odd = rng.random(ctx) < share
        w[b, odd] = np.where(rng.random(odd.sum()) < 0.5, np.nan, -np.inf)
    budget, sink, recent = 300, 5, 20
    lens_d = torch.from_numpy(lens.astype(np.int32)).cuda()
    keep, n = api.kv_evict_select(torch.from_numpy(w).cuda(), lens_d, budget, sink=sink,
                                  recent=recent)
    for b in range(B):
        want = ref.evict(w[b], int(lens[b]), budget, sink, recent)
        assert int(n[b]) == len(want), b
        assert keep[b].tolist() == want + [-1] * (budget - len(want)), b


# ------------------------------------------------------------------ the example


def test_the_example_counts_what_an_eviction_kept(api):
    """A request whose weights are no numbers keeps its sink and recent tokens
    only; the host's lengths and pages are the device's."""
    spec = importlib.util.spec_from_file_location(
        "sparse_decode_kv4", os.path.join(ROOT, "examples", "sparse_decode_kv4.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    d = m.SparseDecoder(2, num_blocks=10, block_size=16, heads=8, kv_heads=2, topk=24, limit=64,
                        budget=40, sink=2, recent=8)

    def rand(*shape):
        return torch.randn(*shape, device="cuda").bfloat16()

    evicted = False
    for step in range(80):
        if step == 63:
            d.key_weights[1] = float("nan")
        d.step(rand(2, 64, 128), torch.rand(2, 64, device="cuda"), rand(2, 128), rand(2, 8, 128),
               rand(2, 2, 128), rand(2, 2, 128))
        assert d.lens == d.context_lens.tolist()
        assert [len(p) for p in d.pages] == [-(-L // 16) for L in d.lens]
        evicted |= d.lens == [40, 10]
    assert evicted
    assert sorted(d.free + [x for p in d.pages for x in p]) == list(range(10))


@pytest.mark.parametrize("rows", [1, 8, 16, 24, 64])
@pytest.mark.parametrize("lens", [[131071], [65536, 30001, 1]])
def test_outputs_over_long_contexts(api, rows, lens):
    """Every channel of contexts up to 131071 keys; what fp16 cannot hold of a
    term is 2^-28 of the largest weight and value."""
    D = 128
    rng = np.random.default_rng(rows)
    kc = [rng.integers(125, 129, size=(L, 1, 4)) for L in lens]
    vc = [rng.integers(124, 129, size=(L, 1, 4)) for L in lens]
    q = rng.standard_normal((len(lens) * rows, D))
    c = Cache(lens, 1, rows, 1, D, 64, kc, vc, q, seed=rows)
    out, lse = api.kv4_attention(*c.args, next_n=1, softmax_scale=0.1)
    for b in range(len(lens)):
        check_row(c, out, lse, b, 0, 0.1, under=2.0 ** -28)
