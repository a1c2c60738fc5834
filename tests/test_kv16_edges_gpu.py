"""The 16-bit cache at the ends of what its calls allow: pages that no token
sees, values that are no numbers, scales and windows of any size."""
import math

import pytest
import torch

from test_kv16_gpu import call, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from top_selection_dsa_gb300 import api as _api
    assert _api.last_device_error() == _api.DSA_OK
    yield _api
    assert _api.last_device_error() == _api.DSA_OK


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
