"""The Python binding of the 4-bit cache's calls, as far as it needs no GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def api():
    from top_selection_dsa_gb300 import build
    build.build()
    from top_selection_dsa_gb300 import api as _api
    return _api


@pytest.mark.parametrize("name", ["kv_evict_workspace_bytes", "kv4_attention_workspace_bytes"])
def test_workspace_sizes_are_asked_for_by_device(api, monkeypatch, name):
    asked = []
    args = dict(kv_evict_workspace_bytes=(3, 640, 64),
                kv4_attention_workspace_bytes=(3, 1, 8, 2, 128, 640))[name]
    helper = dict(kv_evict_workspace_bytes="_evict_workspace",
                  kv4_attention_workspace_bytes="_kv4_workspace")[name]
    monkeypatch.setattr(api, helper, lambda device, *a: asked.append(device) or device)
    monkeypatch.setattr(api.torch.cuda, "is_available", lambda: True)
    for device in (5, 6, 5):
        monkeypatch.setattr(api.torch.cuda, "current_device", lambda: device)
        assert getattr(api, name)(*args) == device
    assert asked == [5, 6, 5]


@pytest.mark.parametrize("planes,row", [(1 << 20, 1 << 19), (1 << 24, 1 << 15), (3, (1 << 31) - 4),
                                        ((1 << 31) - 1, 4)])
def test_compaction_counts_its_work_past_32_bits(api, planes, row):
    """Caches of more slices than a launch takes are refused, also where 32 bits
    would count them to none.  (3 planes of one row of 2 GB are within it.)"""
    A = ctypes.c_void_p(0x10000)
    caches = (api.PagedRows * 1)(api.PagedRows(0x10000, planes, row))
    st = api.lib.dsa_kv_compact(caches, 1, 4, 8, A, 1, None, 0, A, A, A, 0, 8, None, None, 0, None)
    slices = planes * (-(-row // 128))
    assert st == (api.DSA_ERR_UNSUPPORTED if slices > 1 << 30 else api.DSA_OK)
