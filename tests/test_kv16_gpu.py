"""The 16-bit paged cache on the GPU against its definitions in 64 bits:
attention of chunks of new tokens (dsa_kv_attention)."""
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


def make(news, lens, Hq, Hkv, D, block, seed=0, extra=0, strided=False):
    g = torch.Generator().manual_seed(seed)
    table, nblk = ref.pages(g, lens, block, "cuda")
    gd = torch.Generator(device="cuda").manual_seed(seed)
    kc = torch.randn(nblk, Hkv, block, D, generator=gd, device="cuda").bfloat16()
    vc = torch.randn(nblk, Hkv, block, D, generator=gd, device="cuda").bfloat16()
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    T = starts[-1] + extra
    q = (2 * torch.randn(T, Hq + 2 * strided, D, generator=gd, device="cuda")).bfloat16()
    if strided:
        q = q[:, 1:1 + Hq]
    return dict(q=q, kc=kc, vc=vc, table=table, lens=lens, starts=starts,
                lens_d=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                starts_d=torch.tensor(starts, dtype=torch.int32, device="cuda"))


def call(api, s, **kw):
    return api.kv_attention(s["q"], s["kc"], s["vc"], s["table"], s["lens_d"], s["starts_d"], **kw)


def check(s, out, lse, scale=None, window=0, sink=0):
    D = s["q"].shape[-1]
    o, z, tol, ltol = ref.attention(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["starts"],
                                    D ** -0.5 if scale is None else scale, window, sink)
    n = s["starts"][-1]
    for got, want, t in ((out[:n].double(), o[:n], tol[:n]), (lse[:n].double(), z[:n], ltol[:n])):
        fine = torch.isfinite(want)
        assert bool((torch.isfinite(got) == fine).all())
        assert bool((got[~fine].nan_to_num(5.0) == want[~fine].nan_to_num(5.0)).all())
        worst = ((got - want).abs() / t)[fine]
        assert worst.numel() == 0 or worst.max().item() <= 1.0, worst.max().item()


CASES = {
    # news, contexts, Hq, Hkv, D, block
    "one_key": ([1], [1], 8, 1, 128, 64),
    "one_token": ([1], [777], 64, 8, 128, 64),
    "two_tokens_d64": ([2], [130], 4, 4, 64, 8),
    "whole_prompt": ([200], [200], 8, 2, 128, 16),
    "tall_exact": ([32], [128], 8, 1, 128, 128),
    "tall_and_short": ([37], [300], 8, 1, 128, 32),
    "group_5": ([61, 3], [400, 129], 10, 2, 128, 64),
    "group_7_d64": ([100], [1000], 7, 1, 64, 32),
    "group_12": ([25, 1, 30], [256, 255, 31], 24, 2, 128, 8),
    "group_64": ([1, 3, 9], [640, 65, 2000], 64, 1, 128, 64),
    "group_100": ([4], [500], 100, 1, 128, 64),
    "group_128": ([3], [129], 128, 1, 64, 64),
    "heads_16_d64": ([1, 300, 17], [4096, 300, 1000], 16, 16, 64, 16),
    "ragged": ([1, 0, 5, 130, 1, 64, 0], [128, 50, 5, 1000, 1, 64, 0], 16, 4, 128, 64),
    "decode": ([1] * 40, [1 + 97 * i for i in range(40)], 16, 2, 128, 32),
    "long_axis": ([1], [40000], 8, 1, 128, 64),
    "long_axis_tall": ([40], [20000], 8, 1, 128, 64),
    "many_tiles": ([1500], [1500], 8, 8, 64, 64),
}


@pytest.mark.parametrize("name", CASES)
def test_attention(api, name):
    news, lens, Hq, Hkv, D, block = CASES[name]
    s = make(news, lens, Hq, Hkv, D, block, seed=len(name))
    check(s, *call(api, s))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sink", [(1, 0), (100, 0), (128, 4), (300, 130), (257, 1000),
                                         (5000, 4), (1, 1)])
def test_window(api, window, sink, D):
    s = make([1, 200, 40, 1, 3], [1500, 700, 2500, 90, 129], 8, 2, D, 32, seed=window + sink)
    check(s, *call(api, s, window=window, sink=sink), window=window, sink=sink)


@pytest.mark.parametrize("block", [8, 16, 32, 64, 128])
def test_pages(api, block):
    s = make([3, 70], [1000, 333], 8, 2, 128, block, seed=block)
    check(s, *call(api, s))


@pytest.mark.parametrize("window,sink", [(0, 0), (300, 130)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("block", [8, 16])
def test_small_pages(api, block, D, window, sink):
    """Rings that go round many times, tiles cut between SMs, odd key tiles."""
    s = make([1, 260, 37, 2], [9001, 2500, 1283, 8], 12, 3, D, block, seed=block + D)
    check(s, *call(api, s, window=window, sink=sink), window=window, sink=sink)


def test_positions_below_zero_see_nothing(api):
    """Contexts shorter than the new tokens: the first rows are empty."""
    s = make([20, 5, 90, 2], [7, 0, 60, 2], 8, 2, 128, 16, seed=3)
    out, lse = call(api, s)
    check(s, out, lse)
    assert not out[:13].any() and (lse[:13] == -math.inf).all()
    assert not out[20:25].any() and (lse[20:25] == -math.inf).all()


@pytest.mark.parametrize("scale", [2.0 ** -64, 1e-3, 3.0])
def test_scales(api, scale):
    s = make([3, 50], [700, 90], 8, 2, 128, 64, seed=4)
    check(s, *call(api, s, softmax_scale=scale), scale=scale)


def test_growing_and_huge_logits(api):
    """Later keys far above earlier ones: the reference maximum moves many times."""
    s = make([1, 90], [3000, 2000], 8, 1, 128, 64, seed=5)
    for b, L in enumerate(s["lens"]):
        for c in range(L):
            s["kc"][s["table"][b, c // 64].item(), :, c % 64] *= 1 + c / 50
    check(s, *call(api, s))


def test_rows_of_no_request_stay(api):
    s = make([3, 30], [300, 60], 8, 2, 128, 64, seed=6, extra=9)
    out = torch.full_like(s["q"], 7.0)
    lse = torch.full(s["q"].shape[:2], 7.0, device="cuda")
    call(api, s, out=out, lse=lse)
    check(s, out, lse)
    assert (out[33:] == 7).all() and (lse[33:] == 7).all()


def test_strided_queries(api):
    s = make([3, 40], [300, 60], 8, 2, 128, 64, seed=7, strided=True)
    assert not s["q"].is_contiguous()
    check(s, *call(api, s))


def put(s, name, b, c, h, d, x):
    bs = s["kc"].shape[2]
    s[name][s["table"][b, c // bs].item(), h, c % bs, d] = x


@pytest.mark.parametrize("D", [64, 128])
def test_what_a_row_does_not_see_never_reaches_it(api, D):
    """NaN and infinities behind the context, in the future and before the
    window, and among what some rows see."""
    s = make([3, 100, 40], [300, 500, 190], 8, 2, D, 32, seed=8)
    for b, L in enumerate(s["lens"]):
        for c in range(L, s["table"].shape[1] * 32):     # behind the context, in its last page
            if c // 32 < -(-L // 32):
                put(s, "kc", b, c, slice(None), slice(None), math.nan)
                put(s, "vc", b, c, slice(None), slice(None), math.nan)
    put(s, "vc", 0, 299, 0, 5, math.inf)                 # the last row sees these
    put(s, "vc", 1, 450, 1, 6, -math.inf)
    put(s, "vc", 1, 460, 1, 6, math.inf)
    put(s, "vc", 1, 470, 0, slice(None), math.nan)
    put(s, "vc", 2, 170, 1, D - 1, math.nan)
    check(s, *call(api, s))
    put(s, "vc", 1, 100, 1, 3, math.inf)                 # some rows' windows have passed it
    put(s, "vc", 1, 310, 0, 3, math.nan)
    put(s, "kc", 1, 110, 0, 3, math.nan)
    out, lse = call(api, s, window=120, sink=2)
    put(s, "kc", 1, 110, 0, 3, 0.0)                      # no row sees this one
    check(s, out, lse, window=120, sink=2)


def test_seen_nan_keys_and_queries(api):
    s = make([4, 40], [300, 60], 8, 2, 128, 64, seed=9)
    s["q"][2, 3] = math.nan
    put(s, "kc", 1, 50, 1, 0, math.nan)
    out, lse = call(api, s)
    assert out[2, 3].isnan().all() and lse[2, 3].isnan()
    sees = torch.arange(40, device="cuda") + 20 >= 50
    assert out[4:, 4:][sees].isnan().all() and lse[4:, 4:][sees].isnan().all()
    assert not out[4:, 4:][~sees].isnan().any() and not out[4:, :4].isnan().any()
    assert not out[:2].isnan().any() and not out[3].isnan().any()
    assert not out[2, :3].isnan().any() and not out[2, 4:].isnan().any()


def test_same_results_every_time(api):
    s = make([1, 200, 33], [9000, 2000, 400], 16, 2, 128, 64, seed=10)
    a = call(api, s)
    for _ in range(3):
        b = call(api, s)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_graph_reads_its_lengths_when_it_runs(api):
    s = make([40, 50], [1000, 900], 8, 2, 128, 64, seed=11)
    out, lse = call(api, s)
    ws = torch.empty(api.kv_attention_workspace_bytes(90, 8, 2, 128), dtype=torch.uint8,
                     device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(api, s, out=out, lse=lse, workspace=ws)
    for lens, starts in (([1000, 900], [0, 40, 90]), ([130, 64], [0, 1, 2]), ([555, 3], [0, 88, 90])):
        s["lens"], s["starts"] = lens, starts
        s["lens_d"].copy_(torch.tensor(lens))
        s["starts_d"].copy_(torch.tensor(starts))
        graph.replay()
        check(s, out, lse)


def test_two_streams(api):
    sets = [make([1, 70], [5000, 300], 8, 2, 128, 64, seed=i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for s, st in zip(sets, streams):
        with torch.cuda.stream(st):
            got.append([call(api, s) for _ in range(4)])
    torch.cuda.synchronize()
    for s, outs in zip(sets, got):
        for o in outs:
            check(s, *o)


def test_bad_entries_are_recorded(api):
    s = make([2, 20], [300, 200], 8, 2, 128, 64, seed=12)
    good = call(api, s)
    assert api.last_device_error() == api.DSA_OK
    for name, change in (("table", (1, 1, 9999)), ("table", (1, 0, -1)), ("lens_d", (1, 1 << 20)),
                         ("lens_d", (1, -5)), ("starts_d", (2, 23)), ("starts_d", (2, 1))):
        was = s[name].clone()
        s[name][change[:-1]] = change[-1]
        out, lse = call(api, s)
        assert api.last_device_error() == api.DSA_ERR_INVALID_ARG, (name, change)
        assert torch.equal(out[:2], good[0][:2]), (name, change)   # the other request's
        s[name] = was
    again = call(api, s)
    assert api.last_device_error() == api.DSA_OK
    assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])


def test_no_requests_and_no_tokens(api):
    s = make([2], [30], 8, 2, 128, 64)
    out, lse = api.kv_attention(s["q"][:0], s["kc"], s["vc"], s["table"], s["lens_d"],
                                torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8)
    api.kv_attention(s["q"], s["kc"], s["vc"], s["table"][:0], s["lens_d"][:0],
                     s["starts_d"][:1])
