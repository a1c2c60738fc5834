"""The 16-bit cache's operators as a serving loop uses them together: prompts in
chunks beside single tokens, keys rotated into their pages, attention over
them, then an eviction that moves the pages."""
import pytest
import torch

import kv16_reference as ref
from test_kv16_gpu import call, check, make
from test_kv16_rope_gpu import close, rows, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from top_selection_dsa_gb300 import api as _api
    assert _api.last_device_error() == _api.DSA_OK
    yield _api
    assert _api.last_device_error() == _api.DSA_OK


@pytest.mark.parametrize("D,window", [(128, 0), (64, 150)])
def test_serving_loop(api, D, window):
    Hq, Hkv, block, B = 8, 2, 16, 3
    max_blocks = 40
    nblk = B * max_blocks
    table = torch.randperm(nblk, generator=torch.Generator().manual_seed(1)).int() \
        .reshape(B, max_blocks).cuda()
    kc, vc = api.kv_cache(nblk, Hkv, block, D)
    freq, m = api.rope_frequencies(D, 1e4, scaling="yarn", factor=8.0, original_context=512)
    turns = api.rope_turns(freq)
    qw, kw = weights(1, D), weights(2, D)
    lens = [0, 0, 0]
    # request 0: a prompt in chunks; 1: a short prompt, then single tokens; 2 joins late
    for step, news in enumerate([(200, 5, 0), (150, 1, 70), (1, 1, 130), (1, 1, 1), (1, 1, 1)]):
        T = sum(news)
        starts = [0]
        pos, slot = [], []
        for b, n in enumerate(news):
            starts.append(starts[-1] + n)
            for p in range(lens[b], lens[b] + n):
                pos.append(p)
                slot.append(table[b, p // block].item() * block + p % block)
            lens[b] += n
        qkv = rows(10 + step, T, Hq + 2 * Hkv, D)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        pos = torch.tensor(pos, dtype=torch.int32, device="cuda")
        slot = torch.tensor(slot, device="cuda")
        _, _, qr = api.kv_append(k, v, slot, kc, vc, positions=pos, turns=turns, k_weight=kw,
                                 rope_scale=m, q=q, q_weight=qw)
        close(qr, *ref.norm_rope(q, pos, freq, qw, scale=m))
        want, tol = ref.norm_rope(k, pos, freq, kw, scale=m)
        close(kc[slot // block, :, slot % block], want, tol)
        assert torch.equal(vc[slot // block, :, slot % block], v)
        s = dict(q=qr, kc=kc, vc=vc, table=table, lens=list(lens), starts=starts,
                 lens_d=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 starts_d=torch.tensor(starts, dtype=torch.int32, device="cuda"))
        out, lse = call(api, s, window=window, sink=4)
        check(s, out, lse, window=window, sink=4)
    # every request down to 64 tokens, its first 4 and last 32 among them
    kept = torch.rand(B, max_blocks * block, generator=torch.Generator().manual_seed(2)).cuda()
    keep, new_lens = api.kv_evict_select(kept, s["lens_d"], 64, sink=4, recent=32)
    before = [ref.context(c, table, b, L) for c in (kc, vc) for b, L in enumerate(lens)]
    api.kv_compact([kc, vc], keep, s["lens_d"], table, new_lens=new_lens)
    lens2 = new_lens.tolist()
    for i, (c, b) in enumerate((c, b) for c in (kc, vc) for b in range(B)):
        assert torch.equal(ref.context(c, table, b, lens2[b]),
                           before[i][keep[b, :lens2[b]].long()])
    s.update(lens=lens2, lens_d=new_lens)
    check(s, *call(api, s))


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 64)])
def test_most_requests(api, Hq, Hkv, D):
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 40, (2048,), generator=g).tolist()
    news = [min(L, int(n)) for L, n in zip(lens, torch.randint(0, 3, (2048,), generator=g))]
    s = make(news, lens, Hq, Hkv, D, 8, seed=4)
    out, lse = call(api, s)
    # the reference request by request is slow: a few of them
    for b in list(range(0, 2048, 97)) + [2047]:
        t = slice(s["starts"][b], s["starts"][b + 1])
        part = dict(s, q=s["q"][t], table=s["table"][b:b + 1], lens=[lens[b]],
                    starts=[0, news[b]])
        check(part, out[t], lse[t])


def test_pages_past_32_bits(api):
    """A cache of more than 2^32 elements, pages at its far end."""
    D, Hkv, block = 128, 4, 64
    nblk = (1 << 32) // (D * Hkv * block) + 40
    kc = torch.empty(nblk, Hkv, block, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    L = 300
    table = torch.arange(nblk - 1, nblk - 6, -1, dtype=torch.int32, device="cuda")[None]
    p = torch.arange(L, device="cuda")
    slot = table[0].long()[p // block] * block + p % block
    k, v = rows(1, L, Hkv, D), rows(2, L, Hkv, D)
    api.kv_append(k, v, slot, kc, vc)
    assert torch.equal(kc[slot // block, :, slot % block], k)
    assert torch.equal(vc[slot // block, :, slot % block], v)
    s = dict(q=rows(3, 50, 8, D).contiguous(), kc=kc, vc=vc, table=table, lens=[L],
             starts=[0, 50], lens_d=torch.tensor([L], dtype=torch.int32, device="cuda"),
             starts_d=torch.tensor([0, 50], dtype=torch.int32, device="cuda"))
    check(s, *call(api, s))


def test_outputs_of_any_16_byte_alignment(api):
    s = make([3, 40], [300, 60], 8, 2, 128, 64, seed=7)
    room = torch.empty(43 * 8 * 128 + 8, dtype=torch.bfloat16, device="cuda")
    out = room[8:].view(43, 8, 128)
    assert out.data_ptr() % 32 == 16
    lse = torch.empty(43, 8, device="cuda")
    call(api, s, out=out, lse=lse)
    check(s, out, lse)


def test_requests_that_overlap_compute_nothing(api):
    """Starts that go back and forth name more tokens than there are."""
    s = make([1] * 40, [100] * 40, 8, 2, 128, 64, seed=8)
    s["starts_d"].copy_(torch.tensor([0, 40] * 20 + [0]))
    out = torch.full_like(s["q"], 7.0)
    lse = torch.full(s["q"].shape[:2], 7.0, device="cuda")
    call(api, s, out=out, lse=lse)
    assert api.last_device_error() == api.DSA_ERR_INVALID_ARG
    assert (out == 7).all() and (lse == 7).all()
