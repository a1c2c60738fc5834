"""The Python binding of the 4-bit cache's calls, as far as it needs no GPU."""
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
