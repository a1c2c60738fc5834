"""The sparse decode example against plain 64-bit attention over a record of
every token: outputs on the columns it selected, and what evictions keep."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import kv4_reference as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location(
        "sparse_decode_kv4", os.path.join(ROOT, "examples", "sparse_decode_kv4.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_decode_with_evictions_follows_the_plain_computation(example):
    B, Hq, Hkv, D = 2, 8, 2, 128
    d = example.SparseDecoder(B, num_blocks=12, block_size=16, heads=Hq, kv_heads=Hkv, topk=24,
                              limit=64, budget=40, sink=2, recent=8)
    g = torch.Generator(device="cuda").manual_seed(3)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()

    tokens = [[] for _ in range(B)]             # (decoded key, decoded value) in the cache's order
    weight = [np.zeros(0) for _ in range(B)]
    evictions = []
    plain_evict = d.evict

    def evict():
        keep = plain_evict()
        evictions.append(keep.cpu().numpy())
        return keep

    d.evict = evict
    for _ in range(150):
        q, k, v = rand(B, Hq, D), rand(B, Hkv, D), rand(B, Hkv, D)
        n_before = len(evictions)
        out, columns = d.step(rand(B, 64, 128), torch.rand(B, 64, generator=g, device="cuda"),
                              rand(B, 128), q, k, v)
        out, columns = out.double().cpu().numpy(), columns.cpu().numpy()
        for b in range(B):
            dec = []
            for x in (k, v):
                codes, sc = ref.encode(x[b].double().cpu().numpy())
                dec.append(codes), dec.append(sc)
            K, V = ref.decode(ref.pack(dec[0], dec[2]), np.concatenate([dec[1], dec[3]], -1))
            tokens[b].append((K, V))
            weight[b] = np.append(weight[b], 0.0)
            Ks = np.stack([t[0] for t in tokens[b]])
            Vs = np.stack([t[1] for t in tokens[b]])
            o, _, w, (A, Bd) = ref.attention(q[b].double().cpu().numpy(), Ks, Vs, D ** -0.5,
                                             len(tokens[b]), cols=columns[b])
            # fp16 weights, bf16 output and the logits' rounding, as in test_kv4_gpu.py
            tol = A * (2.0 ** -11 + 2.0 ** -17 * Bd[:, None] + 2.0 ** -18) + 2.0 ** -8 * np.abs(o) \
                + 24 * 2.0 ** -24 * np.abs(Vs).max()
            assert (np.abs(out[b] - o) <= tol).all()
            sel = columns[b][columns[b] >= 0]
            weight[b][sel] += w[columns[b] >= 0]
            if len(evictions) > n_before:
                keep = evictions[-1][b]
                keep = keep[keep >= 0]
                want = ref.evict(weight[b], len(tokens[b]), 40, 2, 8)
                # the same set, but for weights closer than their error
                diff = set(keep.tolist()) ^ set(want)
                assert all(abs(weight[b][i] - weight[b][j]) < 1e-4
                           for i in diff for j in diff), diff
                assert np.array_equal(keep[:2], [0, 1]) and len(keep) == 40
                tokens[b] = [tokens[b][i] for i in keep]
                weight[b] = weight[b][keep]
    assert len(evictions) >= 4
    for b in range(B):                          # what is in the cache now
        pos = np.arange(len(tokens[b]))
        slots = torch.tensor([d.pages[b][i // 16] * 16 + i % 16 for i in pos], device="cuda")
        k, v = example.api.kv4_gather(d.cache, d.scales, slots)
        assert np.array_equal(k.double().cpu().numpy(), np.stack([t[0] for t in tokens[b]]))
        assert np.array_equal(v.double().cpu().numpy(), np.stack([t[1] for t in tokens[b]]))
        got = d.key_weights[b].double().cpu().numpy()
        # sums of up to 64 weights of up to 8 heads in fp32, each within 2^-16
        assert np.abs(got[:len(pos)] - weight[b]).max() <= 2.0 ** -16 * 64 * 8
        assert (got[len(pos):] == 0).all()
    assert sorted(d.free + [x for p in d.pages for x in p]) == list(range(12))


def test_the_example_runs(example, capsys):
    example.main(steps=300)
    assert "300 steps" in capsys.readouterr().out
