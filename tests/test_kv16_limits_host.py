"""Limits of the 16-bit cache's calls and the tables they read, on the CPU."""
import math

import pytest
import torch

from test_kv16_abi_host import NUL, api, attend  # noqa: F401  (api: fixture)


@pytest.mark.parametrize("G", [1, 4, 5, 65, 128])
def test_most_work_of_a_call(api, G):
    """(T / (2 floor(128 / G)) + B) (tiles + 3) < 2^30, tiles = the longest
    context's of 128 keys."""
    tiles = (1 << 22) * 64 // 128
    fits = (1 << 30) // (tiles + 3)                      # row tiles
    fits -= fits * (tiles + 3) == 1 << 30
    per = 2 * (128 // G)
    T = (fits - 2) * per
    assert (T // per + 2) * (tiles + 3) < 1 << 30 <= (T // per + 3) * (tiles + 3)
    kw = dict(Hq=G, Hkv=1, qs=G * 128, mb=1 << 22, bs=64, B=2)
    # no workspace: refused for that, behind the limit's check
    assert attend(api, T=T, ws=NUL, **kw) == api.DSA_ERR_INVALID_ARG
    assert attend(api, T=T + per - 1, ws=NUL, **kw) == api.DSA_ERR_INVALID_ARG
    assert attend(api, T=T + per, ws=NUL, **kw) == api.DSA_ERR_UNSUPPORTED


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


def test_stretched_frequencies_between_the_ends(api):
    """Every element from the formula, written out."""
    for rotary, base, factor, ctx, fast, slow in ((64, 1e4, 40.0, 4096, 32, 1),
                                                  (128, 1e6, 4.0, 32768, 32, 1),
                                                  (16, 5e5, 8.0, 8192, 20, 2)):
        freq, m = api.rope_frequencies(rotary, base, scaling="yarn", factor=factor,
                                       original_context=ctx, beta_fast=fast, beta_slow=slow)

        def at(turns):   # base^(-2 i / rotary) ctx / (2 pi) = turns, solved for i
            return rotary / 2 * math.log(ctx / (2 * math.pi * turns), base)

        lo, hi = math.floor(at(fast)), math.ceil(at(slow))
        between = 0
        for i in range(rotary // 2):
            f = base ** (-2 * i / rotary)
            share = min(max((i - lo) / (hi - lo), 0), 1)      # of the divided one
            between += 0 < share < 1
            want = f * (1 - share) + f / factor * share
            assert abs(freq[i].item() - want) <= 1e-13 * want, (rotary, i)
        # the ramp is rotary / 2 log(fast / slow) / log(base) wide: 1.4 elements at least
        assert between >= 1 and abs(m - (1 + math.log(factor) / 10)) < 1e-15


def test_contexts_that_no_element_turns_in(api):
    """An original context so short that even the first element turns less than
    beta_slow times: all are divided."""
    freq, _ = api.rope_frequencies(64, 1e4)
    for kw in (dict(original_context=4), dict(original_context=60, beta_slow=10.0)):
        yarn, _ = api.rope_frequencies(64, 1e4, scaling="yarn", factor=8.0, **kw)
        assert torch.allclose(yarn, freq / 8, rtol=1e-14), kw
