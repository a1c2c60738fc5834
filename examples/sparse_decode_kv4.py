"""Sparse decoding on a 4-bit key/value cache that is held to a budget.

A batch of requests decodes token by token.  Every step

  1. writes the new token's indexer key (LayerNorm, bf16) and its keys and
     values (4 bits) into the request's pages,
  2. lets the indexer select the columns to attend to,
  3. attends to these columns and accumulates their attention weight,

and whenever a request reaches its limit, it is cut down to `budget` tokens by
accumulated weight: the kept rows of the 4-bit cache and of the indexer's keys
move together in place, and the pages behind them are free again.

Run as ``python examples/sparse_decode_kv4.py`` (one GB300; random inputs).
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from top_selection_dsa_gb300 import api  # noqa: E402


class SparseDecoder:
    def __init__(self, batch, num_blocks, *, block_size=64, index_heads=64, heads=32, kv_heads=4,
                 head_dim=128, topk=64, limit=256, budget=128, sink=4, recent=32, device="cuda"):
        self.block_size, self.topk = block_size, topk
        self.limit, self.budget, self.sink, self.recent = limit, budget, sink, recent
        self.max_blocks = -(-limit // block_size)
        self.cache, self.scales = api.kv4_cache(num_blocks, kv_heads, block_size, head_dim, device)
        self.index_keys = torch.zeros(num_blocks, block_size, 128, dtype=torch.bfloat16,
                                      device=device)
        self.ln = torch.ones(128, device=device), torch.zeros(128, device=device)
        # Lengths and pages are known on the host; the device has a copy.
        self.free = list(range(num_blocks))
        self.pages = [[] for _ in range(batch)]
        self.lens = [0] * batch
        self.table = torch.zeros(batch, self.max_blocks, dtype=torch.int32, device=device)
        self.context_lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.key_weights = torch.zeros(batch, self.max_blocks * block_size, device=device)
        width = self.max_blocks * block_size
        self.attn_ws = torch.empty(max(256, api.kv4_attention_workspace_bytes(
            batch, 1, heads, kv_heads, head_dim, topk, selected=True, weights=True)),
            dtype=torch.uint8, device=device)
        self.evict_ws = torch.empty(api.kv_evict_workspace_bytes(batch, width, budget),
                                    dtype=torch.uint8, device=device)

    def step(self, index_q, index_w, index_k, q, k, v):
        """One token of every request: indexer query [B, H, 128], weights
        [B, H] and key [B, 128]; query [B, Hq, D], key and value [B, Hkv, D].
        Returns (attention output like q, selected columns [B, topk])."""
        dev = self.table.device
        slots = []
        for b, L in enumerate(self.lens):
            if L % self.block_size == 0:
                self.pages[b].append(self.free.pop())
                self.table[b, L // self.block_size] = self.pages[b][-1]
            slots.append(self.pages[b][-1] * self.block_size + L % self.block_size)
            self.lens[b] = L + 1
        slots = torch.tensor(slots, device=dev)
        self.context_lens.add_(1)
        api.k_norm_quant_insert(index_k, *self.ln, 1e-6, slots, self.index_keys)
        api.kv4_insert(k, v, slots, self.cache, self.scales)
        columns = api.indexer_topk_paged(index_q, index_w, self.index_keys, self.table,
                                         self.context_lens, self.topk, next_n=1)
        out, _ = api.kv4_attention_topk(q, self.cache, self.scales, self.table, self.context_lens,
                                        columns, next_n=1, key_weights=self.key_weights,
                                        workspace=self.attn_ws)
        if max(self.lens) >= self.limit:
            self.evict()
        return out, columns

    def evict(self):
        keep, new_lens = api.kv_evict_select(self.key_weights, self.context_lens, self.budget,
                                             sink=self.sink, recent=self.recent,
                                             workspace=self.evict_ws)
        api.kv_compact([self.cache, self.scales, self.index_keys], keep, self.context_lens,
                       self.table, new_lens=new_lens, key_weights=self.key_weights)
        self.context_lens = new_lens
        # A request keeps fewer than it could where weights are not numbers.
        self.lens = new_lens.tolist()
        for b in range(len(self.lens)):
            used = -(-self.lens[b] // self.block_size)
            self.free += self.pages[b][used:]
            del self.pages[b][used:]
        return keep


def main(steps=600, batch=4, heads=32, kv_heads=4):
    torch.manual_seed(0)
    d = SparseDecoder(batch, num_blocks=batch * 4, heads=heads, kv_heads=kv_heads)

    def rand(*shape):
        return torch.randn(*shape, device="cuda").bfloat16()

    evicted = 0
    for _ in range(steps):
        before = d.lens[0]
        out, _ = d.step(rand(batch, 64, 128), torch.rand(batch, 64, device="cuda"),
                        rand(batch, 128), rand(batch, heads, 128), rand(batch, kv_heads, 128),
                        rand(batch, kv_heads, 128))
        evicted += before + 1 - d.lens[0]
    torch.cuda.synchronize()
    if api.last_device_error() != api.DSA_OK or not torch.isfinite(out.float()).all():
        raise SystemExit("decode failed")
    print(f"{steps} steps of {batch} requests: {d.lens[0]} tokens each in the cache, "
          f"{evicted} evicted")


if __name__ == "__main__":
    main()
