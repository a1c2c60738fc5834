"""Limits of the 16-bit cache's calls and the tables they read, on the CPU."""
import pytest
import torch

from test_kv16_abi_host import api  # noqa: F401  (fixture)


def test_workspace_of_the_wrong_kind_is_refused(api):
    """A workspace elsewhere than on the call's device, or with gaps, would be
    written past its end."""
    dev = torch.device("cuda", 0)
    for bad in (torch.empty(1000, dtype=torch.uint8),
                torch.empty(1000, dtype=torch.uint8, device="meta")):
        with pytest.raises(ValueError):
            api._workspace(500, dev, bad)
    host = torch.device("cpu")
    with pytest.raises(ValueError):
        api._workspace(500, host, torch.empty(2000, dtype=torch.uint8)[::2])
    with pytest.raises(ValueError):
        api._workspace(500, host, torch.empty(1, dtype=torch.uint8).expand(1000))
    with pytest.raises(ValueError):
        api._workspace(500, host, torch.empty(499, dtype=torch.uint8))
    ok = torch.empty(125, dtype=torch.float32)
    assert api._workspace(500, host, ok) is ok
