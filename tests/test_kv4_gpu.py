"""The 4-bit key/value cache on the GPU against plain 64-bit implementations:
insert and read-back (exact), decode attention over every key and over selected
columns, eviction and compaction (exact).

Tolerances of the attention, from the arithmetic (u = half a step: fp16 2^-11,
bf16 2^-8, fp32 2^-24).  Let B = |scale| max_c sum_d |q_d||k_d| of a row.
  logits   exact fp16 products accumulated in fp32: D/16 tensor-core steps and
           D/32 scaled sums, each within 2^-22 of what it adds to (the tensor
           core truncates), two products with the scale: dS = 2^-19 B covers
           D = 128; q's elements below 2^-24 of the row's largest: another
           2^-24 B.
  weights  e^dS on numerator and sum, ex2 within 2^-21, sums of n terms split
           over 128 lanes and chunks: relative 2 dS + 2^-18.
  output   sum p |V| (2^-11 + 2 dS + 2^-18) + n 2^-24 max|V| (fp16 underflow)
           + 2^-8 |out| (bf16).
"""
import numpy as np
import pytest
import torch

import kv4_reference as ref
from top_selection_dsa_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


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


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def bf16(x):
    """float64 -> (bf16 tensor, its values)."""
    t = torch.from_numpy(np.ascontiguousarray(x)).float().bfloat16()
    return t, t.double().numpy()


# --------------------------------------------------------------- insert, gather


@pytest.mark.parametrize("T,Hkv,D,bs", [(1, 1, 64, 8), (1, 1, 128, 128), (7, 3, 64, 16),
                                        (37, 8, 128, 64), (130, 5, 128, 32), (64, 2, 64, 8)])
def test_insert_writes_the_documented_records(api, T, Hkv, D, bs):
    rng = np.random.default_rng(T * 1000 + D)
    mag = 2.0 ** rng.integers(-20, 20, size=(T, 2 * Hkv, 1))
    kv, val = bf16(rng.standard_normal((T, 2 * Hkv, D)) * mag)
    kv = kv.cuda()
    nb = -(-T // bs) + 2
    cache, scales = api.kv4_cache(nb, Hkv, bs, D)
    slots = rng.permutation(nb * bs)[:T].astype(np.int64)
    api.kv4_insert(kv[:, :Hkv], kv[:, Hkv:], dev(slots), cache, scales)
    kc, ks = ref.encode(val[:, :Hkv])
    vc, vs = ref.encode(val[:, Hkv:])
    want = np.zeros((nb, Hkv, bs, D), np.uint8)
    wsc = np.zeros((nb, Hkv, bs, D // 16), np.uint8)
    want[slots // bs, :, slots % bs] = ref.pack(kc, vc)
    wsc[slots // bs, :, slots % bs] = np.concatenate([ks, vs], -1)
    assert np.array_equal(scales.cpu().numpy(), wsc)
    assert np.array_equal(cache.cpu().numpy(), want)
    k, v = api.kv4_gather(cache, scales, dev(slots))
    wk, wv = ref.decode(ref.pack(kc, vc), np.concatenate([ks, vs], -1))
    assert np.array_equal(k.double().cpu().numpy(), wk)
    assert np.array_equal(v.double().cpu().numpy(), wv)


def test_insert_agrees_with_the_mxfp4_generator(api):
    rng = np.random.default_rng(5)
    x, val = bf16(rng.standard_normal((64, 1, 128)))
    cache, scales = api.kv4_cache(1, 1, 64, 128)
    api.kv4_insert(x.cuda(), x.cuda(), torch.arange(64, device="cuda"), cache, scales)
    packed, sf = wl.quantize_mxfp4_blocks(val[:, 0])
    codes = np.stack([packed & 15, packed >> 4], -1).reshape(64, 128)
    assert np.array_equal(cache.cpu().numpy()[0, 0], ref.pack(codes, codes))
    assert np.array_equal(scales.cpu().numpy()[0, 0], np.concatenate([sf, sf], -1))


def test_insert_special_blocks(api):
    """Zeros, ties, scale boundaries, subnormals, the largest values, NaN and
    infinities (a block of its own each)."""
    D = 128
    rows = np.zeros((8, D))
    rows[0, :7] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]      # with 6: s = 1, all ties
    rows[0, 7] = 6
    rows[0, 32:40] = [-0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6.0]
    rows[1, 0], rows[1, 32], rows[1, 64] = 6.0, 6.03125, 5.96875
    rows[2, 0], rows[2, 32], rows[2, 64] = 2.0 ** -133, 2.0 ** -126, 3 * 2.0 ** -126
    rows[3, 0], rows[3, 33] = 2.0 ** 127, -1.9921875 * 2.0 ** 127
    rows[4, 5], rows[4, 40], rows[4, 70] = np.nan, np.inf, -np.inf
    rows[4, 100] = 1.0
    x, val = bf16(rows[:, None])
    val = val.copy()
    cache, scales = api.kv4_cache(1, 1, 8, D)
    api.kv4_insert(x.cuda(), x.cuda(), torch.arange(8, device="cuda"), cache, scales)
    kc, ks = ref.encode(val)
    assert np.array_equal(scales.cpu().numpy()[0, 0], np.concatenate([ks, ks], -1)[:, 0])
    assert np.array_equal(cache.cpu().numpy()[0, 0], ref.pack(kc, kc)[:, 0])
    k, _ = api.kv4_gather(cache, scales, torch.arange(8, device="cuda"))
    want = torch.from_numpy(ref.decode(ref.pack(kc, kc), np.concatenate([ks, ks], -1))[0])
    assert torch.equal(torch.nan_to_num(k.cpu()), torch.nan_to_num(want.float().bfloat16()))
    assert np.array_equal(np.isnan(k.float().cpu().numpy()), np.isnan(want.numpy()))


def test_insert_skips_padding_and_reports_slots_past_the_cache(api):
    x = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    cache, scales = api.kv4_cache(2, 2, 8, 64)
    api.kv4_insert(x, x, torch.tensor([-1, 3, 16, 15], device="cuda"), cache, scales)
    assert api.last_device_error() == api.DSA_ERR_INVALID_ARG
    used = (scales != 0).any(-1).cpu()
    want = torch.zeros(2, 2, 8, dtype=torch.bool)
    want[0, :, 3] = want[1, :, 7] = True
    assert torch.equal(used, want)
    k, v = api.kv4_gather(cache, scales, torch.tensor([-1, 3, 15], device="cuda"))
    assert (k[0] == 0).all() and (k[1:] == 1).all() and (v[1:] == 1).all()
    api.kv4_gather(cache, scales, torch.tensor([16], device="cuda"))
    assert api.last_device_error() == api.DSA_ERR_INVALID_ARG


# -------------------------------------------------------------------- attention


class Problem:
    """Random queries and cache; pages in random order, what lies outside the
    requests' tokens filled with NaN scales, unused table entries with rubbish."""

    def __init__(self, lens, nn, Hq, Hkv, D, bs, seed=0, qmag=1.5, spread=2):
        rng = np.random.default_rng(seed)
        B = len(lens)
        self.lens, self.nn, self.Hkv, self.D, self.bs = lens, nn, Hkv, D, bs
        nblk = [-(-L // bs) for L in lens]
        total = max(sum(nblk), 1) + 1
        perm = rng.permutation(total)
        mb = max(max(nblk), 1) + 1
        table = rng.choice([-7, 10 ** 9], size=(B, mb)).astype(np.int32)
        rec = rng.integers(0, 256, size=(total, Hkv, bs, D), dtype=np.uint8)
        sc = np.full((total, Hkv, bs, D // 16), 255, np.uint8)
        at = 0
        for b, n in enumerate(nblk):
            table[b, :n] = perm[at:at + n]
            at += n
            for i in range(lens[b]):
                sc[table[b, i // bs], :, i % bs] = rng.integers(
                    127 - spread, 127 + spread + 1, size=(Hkv, D // 16))
        # a head's key scales differ less than its value scales
        self.rec, self.sc, self.table = rec, sc, table
        self.q_t, self.q = bf16(rng.standard_normal((B * nn, Hq, D)) * qmag)
        self.scale = 0.7 * D ** -0.5 / 2.7

    def kv(self, b):
        pos = np.arange(self.lens[b])
        blk, at = self.table[b, pos // self.bs], pos % self.bs
        if len(pos) == 0:
            z = np.zeros((0, self.Hkv, self.D))
            return z, z
        return ref.decode(self.rec[blk, :, at], self.sc[blk, :, at])

    def gpu(self):
        return (self.q_t.cuda(), dev(self.rec), dev(self.sc), dev(self.table),
                dev(np.array(self.lens, np.int32)))


def check(got_out, got_lse, want, V, name):
    out, lse, w, (A, Bd) = want
    n = max(len(w), 1)
    vmax = np.abs(V).max() if V.size else 0.0
    dS = (2.0 ** -19 + 2.0 ** -24) * Bd
    tol = A * (2.0 ** -11 + 2 * dS + 2.0 ** -18)[:, None] + n * 2.0 ** -24 * vmax \
        + 2.0 ** -8 * np.abs(out) + 2.0 ** -140
    err = np.abs(got_out - out)
    assert (err <= tol).all(), (name, float((err - tol).max()), float(err.max()))
    fin = np.isfinite(lse)
    assert np.array_equal(fin, np.isfinite(got_lse)) and (got_lse[~fin] == -np.inf).all(), name
    tl = 2 * dS + 2.0 ** -18 + 2.0 ** -22 * np.abs(np.where(fin, lse, 0))
    assert (np.abs(got_lse - lse)[fin] <= tl[fin]).all(), name
    return 2 * dS.max() + 2.0 ** -18


SHAPES = [  # lens, next_n, Hq, Hkv, D, block
    ([1], 1, 1, 1, 128, 8),
    ([1, 0, 2], 1, 2, 1, 64, 8),
    ([63, 64, 65], 1, 8, 1, 128, 64),
    ([15, 16, 17, 33], 1, 6, 2, 128, 16),
    ([130, 1], 2, 16, 2, 128, 64),
    ([1, 3, 0, 77], 4, 3, 1, 64, 32),          # rows that see nothing
    ([257], 3, 21, 3, 128, 128),               # 7 heads a group, 21 rows: two row tiles
    ([100, 200], 1, 64, 1, 128, 64),           # one shared head, four row tiles
    ([90, 45], 1, 16, 16, 64, 16),             # a head each
    ([1300], 1, 4, 1, 128, 64),                # several chunks
    ([2100, 700, 5], 2, 8, 2, 64, 64),
    ([513, 300], 5, 24, 2, 128, 8),            # 60 rows
    ([300, 77], 2, 16, 2, 64, 16),             # 16 rows, D = 64
    ([300, 1], 1, 24, 1, 64, 32),              # 24 rows, D = 64
    ([520, 3], 2, 32, 1, 64, 64),              # 64 rows, D = 64
    ([200, 129], 2, 96, 2, 128, 64),           # 96 rows: two tiles of 64
    ([6000, 40], 1, 40, 1, 128, 64),           # 40 rows over many CTAs
    ([300] * 40, 1, 2, 1, 64, 16),             # more requests than a warp has lanes
    ([1000, 0, 2, 4000], 3, 11, 1, 128, 32),   # 33 rows, some of which see nothing
]


@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_attention_over_every_key(api, case):
    lens, nn, Hq, Hkv, D, bs = SHAPES[case]
    P = Problem(lens, nn, Hq, Hkv, D, bs, seed=case)
    args = P.gpu()
    out, lse = api.kv4_attention(*args, next_n=nn, softmax_scale=P.scale)
    width = P.table.shape[1] * bs
    acc0 = np.random.default_rng(1).random((len(lens), width + 3)).astype(np.float32)
    acc = dev(acc0)
    out2, lse2 = api.kv4_attention(*args, next_n=nn, softmax_scale=P.scale, key_weights=acc)
    assert torch.equal(out.view(torch.int16), out2.view(torch.int16))
    assert torch.equal(lse, lse2)
    out, lse, acc = out.double().cpu().numpy(), lse.double().cpu().numpy(), acc.cpu().numpy()
    for b, L in enumerate(lens):
        K, V = P.kv(b)
        total, rel = np.zeros(L), 0.0
        for j in range(nn):
            r = b * nn + j
            want = ref.attention(P.q[r], K, V, P.scale, L - nn + j + 1)
            rel = max(rel, check(out[r], lse[r], want, V, (case, r)))
            total += want[2]
        got = acc[b, :L].astype(np.float64) - acc0[b, :L]
        assert (np.abs(got - total) <= rel * total + 2.0 ** -22 * (1 + total)).all(), (case, b)
        assert np.array_equal(acc[b, L:], acc0[b, L:])


@pytest.mark.parametrize("case", range(len(SHAPES)))
@pytest.mark.parametrize("k", [1, 40, 300])
def test_attention_over_selected_columns(api, case, k):
    lens, nn, Hq, Hkv, D, bs = SHAPES[case]
    P = Problem(lens, nn, Hq, Hkv, D, bs, seed=100 + case)
    rng = np.random.default_rng(case * 7 + k)
    sel = np.full((len(lens) * nn, k), -1, np.int32)
    for b, L in enumerate(lens):
        for j in range(nn):
            seen = max(L - nn + j + 1, 0)
            c = rng.permutation(seen)[:k].astype(np.int32)
            if case % 2:                        # holes anywhere, order free
                c = np.where(rng.random(len(c)) < 0.2, -1, c)
            else:
                c = np.sort(c)
            sel[b * nn + j, :len(c)] = c
    args = P.gpu()
    out, lse = api.kv4_attention_topk(*args, dev(sel), next_n=nn, softmax_scale=P.scale)
    sw = torch.full(sel.shape, 7.0, device="cuda")
    width = P.table.shape[1] * bs
    acc = torch.zeros(len(lens), width, device="cuda")
    out2, lse2 = api.kv4_attention_topk(*args, dev(sel), next_n=nn, softmax_scale=P.scale,
                                        sel_weights=sw, key_weights=acc)
    acc3 = torch.zeros(len(lens), width, device="cuda")
    api.kv4_attention_topk(*args, dev(sel), next_n=nn, softmax_scale=P.scale, key_weights=acc3)
    assert torch.equal(out.view(torch.int16), out2.view(torch.int16))
    assert torch.equal(lse, lse2) and torch.equal(acc, acc3)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    sw, acc = sw.double().cpu().numpy(), acc.double().cpu().numpy()
    for b, L in enumerate(lens):
        K, V = P.kv(b)
        total, rel = np.zeros(width), 0.0
        for j in range(nn):
            r = b * nn + j
            want = ref.attention(P.q[r], K, V, P.scale, L - nn + j + 1, cols=sel[r])
            rel = max(rel, check(out[r], lse[r], want, V, (case, k, r)))
            assert (np.abs(sw[r] - want[2]) <= rel * want[2] + 2.0 ** -22 * Hq).all()
            np.add.at(total, sel[r][sel[r] >= 0], want[2][sel[r] >= 0])
        assert (np.abs(acc[b] - total) <= rel * total + 2.0 ** -22 * Hq * nn).all()


def test_selecting_every_key_in_order_is_the_dense_call(api):
    P = Problem([777], 1, 16, 2, 128, 64, seed=3)
    args = P.gpu()
    out, lse = api.kv4_attention(*args, next_n=1, softmax_scale=P.scale)
    sel = torch.arange(777, dtype=torch.int32, device="cuda")[None]
    out2, lse2 = api.kv4_attention_topk(*args, sel, next_n=1, softmax_scale=P.scale)
    # the same sums, cut into the same tiles; only the chunks may differ
    assert torch.allclose(lse, lse2, rtol=2 ** -20, atol=2 ** -18)
    assert torch.allclose(out.float(), out2.float(), rtol=2 ** -6, atol=2 ** -9)


def test_scales_and_queries_of_very_different_size(api):
    """Value scales over 2^+-18 and query rows over 2^+-12 times each other;
    logits stay moderate through softmax_scale and one row of large logits."""
    lens, nn, Hq, Hkv, D, bs = [300], 1, 8, 1, 128, 64
    P = Problem(lens, nn, Hq, Hkv, D, bs, seed=9)
    rng = np.random.default_rng(2)
    G = D // 32
    for i in range(300):
        P.sc[P.table[0, i // bs], :, i % bs, G:] = rng.integers(127 - 18, 127 + 19, size=(Hkv, G))
    mag = 2.0 ** np.array([-12, -6, -3, 0, 1, 2, 3, 5])
    P.q_t, P.q = bf16(P.q[0][None] * mag[None, :, None])
    out, lse = api.kv4_attention(*P.gpu(), next_n=1, softmax_scale=P.scale)
    K, V = P.kv(0)
    want = ref.attention(P.q[0], K, V, P.scale, 300)
    check(out[0].double().cpu().numpy(), lse[0].double().cpu().numpy(), want, V, "spread")


def test_one_query_element_far_above_the_others(api):
    P = Problem([200], 1, 2, 1, 64, 16, seed=11)
    q = P.q.copy()
    q[0, :, 7] = 2.0 ** 14
    q[0, 1] *= 2.0 ** -10
    P.q_t, P.q = bf16(q)
    out, lse = api.kv4_attention(*P.gpu(), next_n=1, softmax_scale=2.0 ** -12)
    K, V = P.kv(0)
    want = ref.attention(P.q[0], K, V, 2.0 ** -12, 200)
    check(out[0].double().cpu().numpy(), lse[0].double().cpu().numpy(), want, V, "far")


def test_nan_values_reach_their_channels_only(api):
    P = Problem([100], 1, 8, 1, 128, 64, seed=12)
    P.sc[P.table[0, 0], 0, 5, 4 + 2] = 255      # value block 2 of token 5
    out, lse = api.kv4_attention(*P.gpu(), next_n=1, softmax_scale=P.scale)
    bad = torch.isnan(out[0]).cpu()
    want = torch.zeros(8, 128, dtype=torch.bool)
    want[:, 64:96] = True
    assert torch.equal(bad, want) and torch.isfinite(lse).all()
    P.sc[P.table[0, 1], 0, 9, 1] = 255          # a key block of token 73
    out, lse = api.kv4_attention(*P.gpu(), next_n=1, softmax_scale=P.scale)
    assert torch.isnan(out).all() and torch.isnan(lse).all()


def test_rows_do_not_see_later_tokens_nan(api):
    """next_n = 2: the last token is NaN throughout; the first row is clean."""
    P = Problem([65], 2, 8, 1, 128, 64, seed=13)
    P.sc[P.table[0, 1], 0, 0] = 255
    out, lse = api.kv4_attention(*P.gpu(), next_n=2, softmax_scale=P.scale)
    assert torch.isfinite(lse[0]).all() and torch.isnan(lse[1]).all()
    assert torch.isfinite(out[0].float()).all() and torch.isnan(out[1].float()).all()


def test_long_cache_offsets_pass_32_bits(api):
    """Pages beyond 2^32 bytes of records."""
    D, Hkv, bs = 128, 8, 64
    nb = (1 << 32) // (Hkv * bs * D) + 40
    cache = torch.zeros(nb, Hkv, bs, D, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(nb, Hkv, bs, D // 16, dtype=torch.uint8, device="cuda")
    x = torch.randn(150, Hkv, D, device="cuda").bfloat16()
    y = torch.randn(150, Hkv, D, device="cuda").bfloat16()
    pages = torch.tensor([nb - 1, nb - 30, nb - 3], device="cuda")
    slots = pages[torch.arange(150, device="cuda") // bs] * bs + \
        torch.arange(150, device="cuda") % bs
    api.kv4_insert(x, y, slots, cache, scales)
    q = torch.randn(1, 16, D, device="cuda").bfloat16()
    lens = torch.tensor([150], dtype=torch.int32, device="cuda")
    out, lse = api.kv4_attention(q, cache, scales, pages.int()[None], lens, next_n=1)
    small, ssc = cache[pages].contiguous(), scales[pages].contiguous()
    table = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    out2, lse2 = api.kv4_attention(q, small, ssc, table, lens, next_n=1)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    k, _ = api.kv4_gather(cache, scales, slots)
    k2, _ = api.kv4_gather(small, ssc, torch.arange(150, device="cuda"))
    assert torch.equal(k, k2)


def test_results_repeat_and_run_on_a_side_stream(api):
    P = Problem([3000, 40], 2, 16, 2, 128, 64, seed=14)
    args = P.gpu()
    acc = torch.zeros(2, P.table.shape[1] * 64, device="cuda")
    out, lse = api.kv4_attention(*args, next_n=2, key_weights=acc)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        acc2 = torch.zeros_like(acc)
        out2, lse2 = api.kv4_attention(*args, next_n=2, key_weights=acc2)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and torch.equal(acc, acc2)


# --------------------------------------------------------- eviction, compaction


@pytest.mark.parametrize("lens,budget,sink,recent,bs", [
    ([1], 1, 0, 0, 8), ([0, 1, 5, 64], 16, 2, 4, 8), ([100, 37, 200], 50, 4, 13, 16),
    ([100, 37, 200], 50, 25, 25, 16), ([300, 999], 128, 0, 0, 64), ([1000, 3], 600, 4, 32, 64),
    ([20000, 17000], 700, 4, 64, 64),
])
def test_evict_select_and_compact(api, lens, budget, sink, recent, bs):
    rng = np.random.default_rng(budget + len(lens))
    B = len(lens)
    nblk = [-(-L // bs) for L in lens]
    keepn = [min(budget, L) for L in lens]
    newb = [-(-n // bs) for n in keepn]
    total = sum(nblk) + sum(newb) + 1
    perm = rng.permutation(total)
    mb, mn = max(max(nblk), 1), max(max(newb), 1)
    table = np.full((B, mb), -9, np.int32)
    fresh = np.full((B, mn), -9, np.int32)
    at = 0
    for b in range(B):
        table[b, :nblk[b]] = perm[at:at + nblk[b]]
        at += nblk[b]
    for b in range(B):
        fresh[b, :newb[b]] = perm[at:at + newb[b]]
        at += newb[b]
    ldw = mb * bs
    w = np.round(rng.random((B, ldw)) * 40).astype(np.float32) / 8        # many ties
    for b, L in enumerate(lens):
        w[b, L:] = 1e9                          # beyond the request: never looked at
    w0 = w.copy()
    cl = dev(np.array(lens, np.int32))
    keep, new_lens = api.kv_evict_select(dev(w), cl, budget, sink=sink, recent=recent)
    want = [ref.evict(w[b], L, budget, sink, recent) for b, L in enumerate(lens)]
    assert new_lens.tolist() == [len(x) for x in want]
    for b in range(B):
        assert keep[b].tolist() == want[b] + [-1] * (budget - len(want[b]))
    caches = [rng.integers(0, 256, size=s, dtype=np.uint8) for s in
              ((total, 3, bs, 128), (total, 3, bs, 8), (total, bs, 256), (total, bs, 4),
               (total, 2, bs, 12), (total, bs, 200))]
    for in_place in (False, True):
        gpu = [dev(c) for c in caches]
        weights = dev(w0)
        out = weights if in_place else torch.full_like(weights, 3.0)
        api.kv_compact(gpu, keep, cl, dev(table), None if in_place else dev(fresh),
                       new_lens=new_lens, key_weights=weights, key_weights_out=out)
        for c, g in zip(caches, gpu):
            exp = c.copy()
            for b in range(B):
                for i, pos in enumerate(want[b]):
                    tab = table if in_place else fresh
                    src = (table[b, pos // bs], slice(None), pos % bs) if c.ndim == 4 else \
                        (table[b, pos // bs], pos % bs)
                    dst = (tab[b, i // bs], slice(None), i % bs) if c.ndim == 4 else \
                        (tab[b, i // bs], i % bs)
                    exp[dst] = c[src]
            assert np.array_equal(g.cpu().numpy(), exp), (c.shape, in_place)
        ew = np.zeros_like(w0)
        for b in range(B):
            ew[b, :len(want[b])] = w0[b, want[b]]
        assert np.array_equal(out.cpu().numpy(), ew)


def test_evict_never_keeps_nan_or_minus_infinity(api):
    w = np.ones((1, 64), np.float32)
    w[0, 10:20] = np.nan
    w[0, 20:30] = -np.inf
    w[0, 30] = np.inf
    keep, n = api.kv_evict_select(dev(w), dev(np.array([64], np.int32)), 60, sink=2, recent=3)
    assert n.tolist() == [44]
    assert keep[0, :44].tolist() == list(range(10)) + list(range(30, 64))
    assert (keep[0, 44:] == -1).all()


def test_compact_weights_in_place_with_fresh_pages(api):
    """The weights rewritten where they lie while the rows go to new pages,
    with more rows than one CTA takes."""
    bs, L, budget = 64, 6400, 5000
    rng = np.random.default_rng(8)
    w = rng.random((1, L)).astype(np.float32)
    table = np.arange(100, dtype=np.int32)[None]
    fresh = np.arange(100, 200, dtype=np.int32)[None]
    cache = rng.integers(0, 256, size=(200, bs, 16), dtype=np.uint8)
    g, wg, cl = dev(cache), dev(w), dev(np.array([L], np.int32))
    keep, n = api.kv_evict_select(wg, cl, budget, sink=1, recent=1)
    api.kv_compact([g], keep, cl, dev(table), dev(fresh), new_lens=n, key_weights=wg)
    pos = np.array(ref.evict(w[0], L, budget, 1, 1))
    want = np.zeros_like(w)
    want[0, :budget] = w[0, pos]
    assert np.array_equal(wg.cpu().numpy(), want)
    flat = cache.reshape(-1, 16)
    got = g.cpu().numpy().reshape(-1, 16)
    assert np.array_equal(got[6400:6400 + budget], flat[pos])
    assert np.array_equal(got[:6400], flat[:6400])


# --------------------------------------------------------- bad device-side values


def test_bad_pages_lengths_and_columns_are_recorded(api):
    P = Problem([100, 50], 1, 8, 1, 128, 64, seed=15)
    q, rec, sc, table, cl = P.gpu()
    sc = torch.where(sc == 255, torch.full_like(sc, 127), sc)
    bad = table.clone()
    bad[0, 1] = rec.shape[0]
    out, lse = api.kv4_attention(q, rec, sc, bad, cl, next_n=1)
    assert api.last_device_error() == api.DSA_ERR_INVALID_ARG
    zero = table.clone()
    zero[0, 1] = 0
    out2, lse2 = api.kv4_attention(q, rec, sc, zero, cl, next_n=1)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    long = cl.clone()
    long[1] = -4
    out, lse = api.kv4_attention(q, rec, sc, table, long, next_n=1)
    assert api.last_device_error() == api.DSA_ERR_INVALID_ARG
    assert (out[1] == 0).all() and (lse[1] == -torch.inf).all()
    sel = torch.tensor([[3, 100, -2, 99], [0, 1, 49, -1]], dtype=torch.int32, device="cuda")
    out, lse = api.kv4_attention_topk(q, rec, sc, table, cl, sel, next_n=1)
    assert api.last_device_error() == api.DSA_ERR_INVALID_ARG
    sel[0] = torch.tensor([3, -1, -1, 99])
    out2, lse2 = api.kv4_attention_topk(q, rec, sc, table, cl, sel, next_n=1)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_compact_skips_bad_entries(api):
    bs = 8
    g = torch.arange(4 * bs, dtype=torch.int32, device="cuda").reshape(4, bs).clone()
    before = g.clone()
    keep = torch.tensor([[0, 5, 40, 9]], dtype=torch.int32, device="cuda")
    cl = torch.tensor([16], dtype=torch.int32, device="cuda")
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    fresh = torch.tensor([[3]], dtype=torch.int32, device="cuda")
    n = torch.tensor([4], dtype=torch.int32, device="cuda")
    api.kv_compact([g], keep, cl, table, fresh, new_lens=n)
    assert api.last_device_error() == api.DSA_ERR_INVALID_ARG
    want = before.clone()
    want[3, 0], want[3, 1], want[3, 3] = before[0, 0], before[0, 5], before[1, 1]
    assert torch.equal(g, want)
    fresh[0, 0] = 9
    api.kv_compact([g], keep[:, :2].contiguous(), cl, table, fresh,
                   new_lens=torch.tensor([2], dtype=torch.int32, device="cuda"))
    assert api.last_device_error() == api.DSA_ERR_INVALID_ARG
    assert torch.equal(g, want)


# ----------------------------------------------------------------------- graphs


def test_a_decode_step_in_a_graph(api):
    """Insert, attention with accumulated weights, selected attention: captured
    once, replayed with other lengths and inputs."""
    P = Problem([500, 77], 1, 16, 2, 128, 64, seed=16)
    q, rec, sc, table, cl = P.gpu()
    table = torch.where((table < 0) | (table >= rec.shape[0]), torch.zeros_like(table), table)
    new = torch.randn(2, 2, 128, device="cuda").bfloat16()
    slots = torch.tensor([int(table[0, 7]) * 64 + 51, int(table[1, 1]) * 64 + 12], device="cuda")
    sel = torch.stack([torch.arange(60, dtype=torch.int32, device="cuda")] * 2)
    acc = torch.zeros(2, table.shape[1] * 64, device="cuda")

    def step():
        api.kv4_insert(new, new, slots, rec, sc)
        a = api.kv4_attention(q, rec, sc, table, cl, next_n=1, key_weights=acc)
        b = api.kv4_attention_topk(q, rec, sc, table, cl, sel, next_n=1)
        return a, b

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = step()
    for lens in ([500, 77], [300, 60]):
        cl.copy_(torch.tensor(lens))
        q.copy_(torch.randn_like(q))
        acc.zero_()
        g.replay()
        got = [t.clone() for pair in captured for t in pair] + [acc.clone()]
        acc.zero_()
        eager = step()
        for x, y in zip(got, [t for pair in eager for t in pair] + [acc]):
            assert torch.equal(x, y)


# ------------------------------------------- sizes on either side of a variant


@pytest.mark.parametrize("B", [152, 153, 400])
def test_evict_select_of_more_requests_than_sms(api, B):
    rng = np.random.default_rng(B)
    ctx, budget, sink, recent = 900, 200, 4, 30
    lens = [0, 1, 200, 201, ctx] + [int(x) for x in rng.integers(1, ctx, size=B - 5)]
    w = np.exp(3 * rng.standard_normal((B, ctx))).astype(np.float32)
    w[:, ::7] = 0.0
    keep, n = api.kv_evict_select(dev(w), dev(np.array(lens, np.int32)), budget, sink=sink,
                                  recent=recent)
    keep = keep.cpu().numpy()
    for b, L in enumerate(lens):
        want = ref.evict(w[b], L, budget, sink, recent)
        assert int(n[b]) == len(want)
        assert keep[b].tolist() == want + [-1] * (budget - len(want))


@pytest.mark.parametrize("B,ctx", [(2, 32768), (2, 32769), (40, 33000), (1, 131072)])
def test_evict_select_on_either_side_of_the_one_kernel_path(api, B, ctx):
    rng = np.random.default_rng(ctx)
    lens = [ctx] + [int(x) for x in rng.integers(1, ctx, size=B - 1)]
    w = np.exp(3 * rng.standard_normal((B, ctx))).astype(np.float32)
    w[:, ::7] = 0.0
    w[0, 100:5000] = 1.0                        # thousands of ties across the bound
    w[:, 11] = -0.0
    budget, sink, recent = 3000, 4, 100
    keep, n = api.kv_evict_select(dev(w), dev(np.array(lens, np.int32)), budget, sink=sink,
                                  recent=recent)
    for b, L in enumerate(lens):
        want = ref.evict(w[b], L, budget, sink, recent)
        assert int(n[b]) == len(want)
        assert keep[b].tolist() == want + [-1] * (budget - len(want))


@pytest.mark.parametrize("values", ["equal", "two", "zero", "negative"])
@pytest.mark.parametrize("room", [0, 1, 31, 500])
def test_evict_select_few_distinct_weights(api, values, room):
    L = 1500
    w = np.full((1, L), {"equal": 2.5, "two": 1.0, "zero": 0.0, "negative": -3.0}[values],
                np.float32)
    if values == "two":
        w[0, 700:730] = 9.0
    if values == "negative":
        w[0, 3::5] = -1.0
    keep, n = api.kv_evict_select(dev(w), dev(np.array([L], np.int32)), room + 7, sink=3, recent=4)
    want = ref.evict(w[0], L, room + 7, 3, 4)
    assert n.tolist() == [len(want)] and keep[0].tolist() == want


@pytest.mark.parametrize("Hq", [4, 16, 24])
@pytest.mark.parametrize("scale", [0.0, -0.04])
def test_zero_and_negative_softmax_scale(api, Hq, scale):
    P = Problem([150], 1, Hq, 1, 128, 64, seed=21)
    out, lse = api.kv4_attention(*P.gpu(), next_n=1, softmax_scale=scale)
    K, V = P.kv(0)
    want = ref.attention(P.q[0], K, V, scale, 150)
    check(out[0].double().cpu().numpy(), lse[0].double().cpu().numpy(), want, V, scale)


@pytest.mark.parametrize("Hq", [4, 16, 24])
@pytest.mark.parametrize("scale", [1e4, 1e8, 1e12])
def test_huge_logits_pick_the_largest(api, Hq, scale):
    """Logits far apart: the output is one value row, nothing overflows."""
    P = Problem([150], 1, Hq, 1, 128, 64, seed=22, spread=0)
    out, lse = api.kv4_attention(*P.gpu(), next_n=1, softmax_scale=scale)
    K, V = P.kv(0)
    S = np.einsum("hd,ld->hl", P.q[0], K[:, 0])
    best = S.argmax(1)
    second = np.sort(S, 1)[:, -2]
    # the row is alone where the gap is far above the logits' rounding (2^-19 of
    # sum |q||k|) and above 20 in the exponent
    B = (np.abs(P.q[0]) @ np.abs(K[:, 0]).T).max(1)
    alone = (S.max(1) - second > 2.0 ** -17 * B) & ((S.max(1) - second) * scale > 20)
    assert alone.sum() >= 1
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    got = out[0].double().cpu().numpy()
    for h in np.nonzero(alone)[0]:
        assert np.abs(got[h] - V[best[h], 0]).max() <= 2.0 ** -8 * np.abs(V[best[h], 0]).max()


@pytest.mark.parametrize("Hq", [4, 16, 24])
def test_infinite_and_nan_queries_stay_in_their_rows(api, Hq):
    P = Problem([100], 1, Hq, 1, 128, 64, seed=23)
    q, rec, sc, table, cl = P.gpu()
    q[0, 1, 5] = float("nan")
    q[0, 3, 9] = float("inf")
    out, lse = api.kv4_attention(q, rec, sc, table, cl, next_n=1, softmax_scale=P.scale)
    assert torch.isnan(out[0, 1].float()).all() and torch.isnan(lse[0, 1])
    K, V = P.kv(0)
    want = ref.attention(P.q[0], K, V, P.scale, 100)
    keep = [h for h in range(Hq) if h not in (1, 3)]
    check(out[0, keep].double().cpu().numpy(), lse[0, keep].double().cpu().numpy(),
          (want[0][keep], want[1][keep], want[2], (want[3][0][keep], want[3][1][keep])), V, "rows")
