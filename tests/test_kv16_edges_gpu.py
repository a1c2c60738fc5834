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
