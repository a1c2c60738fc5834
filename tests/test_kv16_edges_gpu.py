"""The 16-bit cache at the ends of what its calls allow: pages that no token
sees, values that are no numbers, scales and windows of any size."""
import math

import pytest
import torch

import kv16_reference as ref
from test_kv16_gpu import call, check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from top_selection_dsa_gb300 import api as _api
    assert _api.last_device_error() == _api.DSA_OK
    yield _api
    assert _api.last_device_error() == _api.DSA_OK


@pytest.mark.parametrize("window,sink", [(1, 0), (100, 4), (300, 130), (257, 0)])
@pytest.mark.parametrize("D,block", [(128, 8), (64, 8), (64, 16), (128, 32), (64, 64), (128, 128)])
def test_entries_of_pages_that_no_token_sees(api, D, block, window, sink):
    """Pages behind the window that a serving loop has freed."""
    s = make([1, 200, 40, 1, 3, 1], [1500, 700, 2500, 90, 129, 9001], 8, 2, D, block,
             seed=window + sink)
    table = s["table"].clone()
    gone = 0
    for b, L in enumerate(s["lens"]):
        seen = ref.sees(s["starts"][b + 1] - s["starts"][b], L, window, sink, "cuda").any(0)
        for page in range(-(-L // block)):
            if not seen[page * block:(page + 1) * block].any():
                table[b, page] = -1 if page % 2 else 1 << 30
                gone += 1
    assert gone or block == 128
    out, lse = call(api, dict(s, table=table), window=window, sink=sink)
    assert api.last_device_error() == api.DSA_OK
    check(s, out, lse, window=window, sink=sink)
    # one that a token sees is recorded all the same
    L = s["lens"][1]
    table[1, (L - window) // block] = -1
    call(api, dict(s, table=table), window=window, sink=sink)
    assert api.last_device_error() == api.DSA_ERR_INVALID_ARG


def test_positions_below_zero_look_up_no_page(api):
    s = make([300, 5], [3, 0], 8, 2, 128, 16, seed=3)
    table = s["table"].clone()
    table[1] = -1
    out, lse = call(api, dict(s, table=table))
    assert api.last_device_error() == api.DSA_OK
    check(s, out, lse)


def spoil_tails(s):
    """NaN in the keys and values behind every context, in its last page."""
    bs = s["kc"].shape[2]
    for b, L in enumerate(s["lens"]):
        if L % bs:
            page = s["table"][b, L // bs].item()
            s["kc"][page, :, L % bs:] = math.nan
            s["vc"][page, :, L % bs:] = math.nan


def pass_us(f):
    for _ in range(3):
        f()
    best = math.inf
    for _ in range(8):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(5):
            f()
        b.record()
        b.synchronize()
        best = min(best, 200 * a.elapsed_time(b))
    return best


@pytest.mark.parametrize("news", [1, 20])
def test_values_that_no_row_sees_cost_no_time(api, news):
    """NaN behind the contexts: the same results, bit for bit, and about the
    same time (they are cleared, and nothing looks for them afterwards)."""
    lens = [1000 + 61 * i for i in range(64)]
    s = make([news] * 64, lens, 64, 8, 128, 64, seed=1)
    kw = dict(out=torch.empty_like(s["q"]),
              lse=torch.empty(s["q"].shape[:2], device="cuda"))
    clean = pass_us(lambda: call(api, s, **kw))
    want = [kw["out"].clone(), kw["lse"].clone()]
    spoil_tails(s)
    spoiled = pass_us(lambda: call(api, s, **kw))
    assert torch.equal(kw["out"], want[0]) and torch.equal(kw["lse"], want[1])
    print(f"clean {clean:.1f} us, NaN behind the contexts {spoiled:.1f} us")
    assert spoiled < 1.5 * clean, (spoiled, clean)


@pytest.mark.parametrize("news,L,high", [
    (1, 200, 128), (1, 700, 600), (1, 20000, 600), (1, 20000, 19000), (40, 20000, 600),
    (40, 20000, 19000), (100, 6000, 5000), (3, 131000, 130000)])
def test_seen_values_that_are_no_numbers_and_weigh_nothing(api, news, L, high):
    """Keys from `high` on have logits 200 above the others': what is not finite
    among the values before them has weights of exp(-200), and shows, wherever
    the work is cut."""
    D = 128
    s = make([news], [L], 8, 1, D, 64, seed=2)
    s["q"].fill_(4.0)
    table = s["table"][0].long()
    c = torch.arange(L, device="cuda")
    s["kc"].zero_()
    s["kc"][table[c[high:] // 64], 0, c[high:] % 64] = 200 / (4 * D ** 0.5)

    def put(key, d, x):
        s["vc"][table[key // 64], 0, key % 64, d] = x

    for key in (3, high // 2, high - 1):
        put(key, 5 + key % 3, math.inf)
    put(high // 3, 20, -math.inf)
    put(high // 2, 21, math.nan)
    put(7, 22, math.inf)
    put(high - 2, 22, -math.inf)
    out, lse = call(api, s)
    o, z, tol, ltol = ref.attention(s["q"], s["kc"], s["vc"], s["table"], [L], s["starts"],
                                    D ** -0.5)
    out = out.double()
    assert torch.equal(torch.isfinite(out), torch.isfinite(o))
    fine = torch.isfinite(o)
    assert ((out - o).abs() <= tol)[fine].all()
    # an infinity times a weight that fp32 holds as zero is no number
    assert (out.isnan() | (out == o) | fine).all()
    assert ((lse.double() - z).abs() <= ltol).all()


@pytest.mark.parametrize("scale", [2.0 ** 10, 1e5, 2.0 ** 18, 2.0 ** 21, 3e11, 2.0 ** 64])
@pytest.mark.parametrize("D,news,lens", [(128, [1, 60], [3000, 500]), (64, [1, 200], [9001, 200])])
def test_largest_scales(api, D, news, lens, scale):
    """Logits up to 2^27 count; past 2^28 rows are no numbers, never wrong ones.
    Whole numbers, whose products are exact: what is left is the scale."""
    s = make(news, lens, 8, 2, D, 64, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    for name in ("q", "kc"):
        s[name].copy_(torch.randint(-3, 4, s[name].shape, generator=g, device="cuda"))
    out, lse = call(api, s, softmax_scale=scale)
    scale = torch.tensor(scale, dtype=torch.float32).double().item()
    for b, L in enumerate(lens):
        rows = slice(s["starts"][b], s["starts"][b + 1])
        K, V = (ref.context(s[n], s["table"], b, L).double() for n in ("kc", "vc"))
        ok = ref.sees(news[b], L, 0, 0, "cuda")
        for h in range(8):
            S = s["q"][rows, h].double() @ K[:, h // 4].T
            most = torch.where(ok, S.abs(), 0.0).amax(-1) * scale
            S = S.masked_fill(~ok, -math.inf)
            top = S.amax(-1, keepdim=True)
            w = ((S - top) * scale).exp()
            l = w.sum(-1, keepdim=True)
            want = w / l @ V[:, h // 4]
            size = w / l @ V[:, h // 4].abs()
            # a step of S is 1024 at least, so that weights are 0 or all alike: the
            # output's half step, theirs, the sum's and the division's roundings
            got = out[rows, h].double()
            close = ((got - want).abs() <= ref.BF16 * want.abs() + 1e-38 +
                     (ref.BF16 * (1 + ref.BF16) + (L + 40) * ref.F32) * size).all(-1)
            z = (top * scale + l.log())[:, 0]
            # the logit's product, log(2) and its inverse: a rounding each
            close &= (lse[rows, h].double() - z).abs() <= 8 * ref.F32 * z.abs() + 1e-5
            nan = got.isnan().all(-1) & lse[rows, h].isnan()
            assert (close | nan).all()
            assert close[most <= 2.0 ** 27].all()
            assert nan[top[:, 0] * scale > 2.0 ** 28].all()
    assert api.last_device_error() == api.DSA_OK


@pytest.mark.parametrize("interleaved", [False, True])
def test_angles_near_quarter_turns(api, interleaved):
    """The angle's error is at most 2^-28 turns where a cosine or sine is nearly
    zero too: there it is all that the result consists of."""
    F, D = 32, 64
    near = [24, -24, 5, -5, 40, -100, 1001, -77777]          # units of 2^-32 turns
    whole = [(q << 62) + (n << 32) + 12345 for q in range(4) for n in near]
    turns = torch.tensor([w - 2 ** 64 if w >= 2 ** 63 else w for w in whole], device="cuda")
    q = torch.zeros(1, 1, D)
    q[..., 0::2 if interleaved else 1] = 1.0                 # pairs (1, 0)
    if not interleaved:
        q[..., F:] = 0.0
    pos = torch.ones(1, dtype=torch.int32, device="cuda")
    got, _ = api.qk_norm_rope(q.bfloat16().cuda(), None, pos, turns, interleaved=interleaved)
    got = got[0, 0].double().cpu()
    cos, sin = (got[0::2], got[1::2]) if interleaved else (got[:F], got[F:])
    t = torch.tensor([2 * math.pi * w / 2 ** 64 for w in whole], dtype=torch.float64)
    # half a step of bf16, sincospif's two steps and its products' roundings,
    # and the angle's 2^-28 turns (2 pi / 2^64 in float64: 2^-50)
    rel, angle = ref.BF16 + 8 * ref.F32, 2 * math.pi * 2.0 ** -28 + 2.0 ** -50
    assert ((cos - t.cos()).abs() <= rel * t.cos().abs() + angle * t.sin().abs()).all()
    assert ((sin - t.sin()).abs() <= rel * t.sin().abs() + angle * t.cos().abs()).all()


def test_windows_past_32_bits(api):
    """A window or first tokens of any size that Python holds."""
    s = make([1, 40], [1500, 90], 8, 2, 128, 64, seed=9)
    want = call(api, s)
    for kw in (dict(window=2 ** 31), dict(window=2 ** 32 + 5), dict(window=2 ** 63),
               dict(window=9, sink=2 ** 32 + 1), dict(window=9, sink=2 ** 40)):
        got = call(api, s, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), kw
    for kw in (dict(window=-1), dict(window=-2 ** 32), dict(window=9, sink=-2 ** 40)):
        with pytest.raises(api.DSAError):
            call(api, s, **kw)
