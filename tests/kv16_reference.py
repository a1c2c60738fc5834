"""The 16-bit cache's operators from their definitions, in 64 bits, with the
error bounds that the library's arithmetic allows."""
import math

import torch

BF16 = 2.0 ** -8          # half a step, relative
F32 = 2.0 ** -24


def pages(g, lens, block, device, spare=3):
    """A block table with the blocks in random order, and the block count."""
    need = [max(-(-L // block), 1) for L in lens]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(need)), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table.to(device), total


def context(cache, table, b, L):
    """Request b's first L rows [L, Hkv, D] of a paged cache."""
    bs = cache.shape[2]
    pg = table[b, :-(-L // bs)].long()
    return cache[pg].transpose(1, 2).reshape(-1, cache.shape[1], cache.shape[3])[:L]


def sees(n, L, window, sink, device):
    """[n, L] truth values: what each of the last n positions of L sees."""
    p = torch.arange(L - n, L, device=device)[:, None]
    c = torch.arange(L, device=device)[None]
    ok = c <= p
    if window:
        ok &= (c > p - window) | (c < sink)
    return ok


def attention(q, kc, vc, table, lens, starts, scale, window=0, sink=0):
    """(out, lse, bound of out, bound of lse), float64; rows of no request NaN."""
    T, Hq, D = q.shape
    Hkv = kc.shape[1]
    G = Hq // Hkv
    out = torch.full((T, Hq, D), math.nan, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64, device=q.device)
    ltol = torch.zeros_like(lse)
    for b, L in enumerate(lens):
        t0, n = starts[b], starts[b + 1] - starts[b]
        K = context(kc, table, b, L).double()
        V = context(vc, table, b, L).double()
        ok = sees(n, L, window, sink, q.device)
        for h in range(Hq):
            x = q[t0:t0 + n, h].double()
            k, v = K[:, h // G], V[:, h // G]
            S = (x @ k.T * scale).masked_fill(~ok, -math.inf)
            z = torch.logsumexp(S, -1) if L else torch.full((n,), -math.inf,
                                                           dtype=torch.float64, device=q.device)
            w = torch.exp(S - torch.where(z == -math.inf, 0.0, z)[:, None]).masked_fill(~ok, 0.0)
            bad = ~torch.isfinite(v)
            o = w @ torch.where(bad, 0.0, v)
            # infinities and NaN count where they are seen
            pos = ok.double() @ ((v == math.inf) | v.isnan()).double() > 0
            neg = ok.double() @ ((v == -math.inf) | v.isnan()).double() > 0
            o = torch.where(pos & neg, math.nan, torch.where(pos, math.inf,
                                                            torch.where(neg, -math.inf, o)))
            out[t0:t0 + n, h], lse[t0:t0 + n, h] = o, z
            # A logit: D products summed in fp32 and the scale, its difference
            # from the maximum, the exponential's 2^-22, the sum of L terms
            # (partial sums of 128 columns in four chains, tiles one by one).
            size = torch.where(torch.isfinite(k), k, 0.0).abs()
            S_abs = torch.nan_to_num(x.abs() @ size.T * scale, 0.0, 0.0, 0.0).masked_fill(~ok, 0.0)
            top = S_abs.amax(-1) if L else torch.zeros(n, dtype=torch.float64, device=q.device)
            d = (D + 8) * F32 * top + 2.0 ** -21 + (40 + L / 128) * F32
            A = w @ torch.where(bad, 0.0, v).abs()
            # weights rounded to bf16, the output rounded to bf16
            tol[t0:t0 + n, h] = BF16 * o.abs().nan_to_num(0.0, 0.0, 0.0) + \
                (BF16 * (1 + BF16) + 4 * d[:, None] + (L + 40) * F32) * A + 1e-38
            ltol[t0:t0 + n, h] = 2 * d + 4 * F32 * z.abs().nan_to_num(0.0, 0.0, 0.0)
    return out, lse, tol, ltol


def norm_rope(x, positions, freq, weight=None, eps=1e-6, interleaved=False, scale=1.0):
    """(rows [T, H, D] normalised and rotated, bound of their error), float64.

    The bound: half a bf16 step of the result; fp32 arithmetic of about D/8 + 12
    roundings on the terms' sizes; an angle off by 2^-31 turns and sincospi's
    argument and result by 3 steps of fp32."""
    x = x.double()
    D = x.shape[-1]
    if weight is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    F = 0 if freq is None else freq.numel()
    y, size = x.clone(), x.abs()
    if F:
        t = positions.double().cpu()[:, None] * freq.double().cpu()
        c, s = (t.cos() * scale).to(x.device)[:, None], (t.sin() * scale).to(x.device)[:, None]
        i = torch.arange(F)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + F)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
        both = (x[..., a].abs() + x[..., b].abs()) * abs(scale)
        size[..., a] = both
        size[..., b] = both
    tol = BF16 * y.abs() + ((D / 8 + 12) * F32 + 2 * math.pi * 2.0 ** -31 + 6 * F32) * size
    # float64 angles of large positions are themselves rounded
    if F:
        far = positions.double().abs().max().item() * float(freq.abs().max()) * 2.0 ** -52
        tol = tol + far * size
    return y, tol + 1e-38
