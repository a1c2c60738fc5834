"""The 16-bit paged key/value cache's operators as a user calls them, in plain
form and through this package, over the sizes they are used at.

  rope     queries and keys: a norm of each head and the rotation by position,
           in one pass (qk_norm_rope)
  append   new keys and values written to their pages, keys normalised and
           rotated on the way, the step's queries beside them (kv_append)
  attend   attention of chunks of new tokens over the paged cache, from one
           token a request to whole prompts, with or without a sliding window
           and first tokens that stay visible (kv_attention)

``own`` chooses the side ``run`` takes: False computes in elementary torch
operations in 32 bits (angles in 64), rounded once at the end; True calls the
package.  ``exact`` computes the definitions in 64 bits, apart from both.

Definitions, for a head's row x of D elements at position p:
  norm      y = x / sqrt(mean(x^2) + eps) * weight
  rotation  of the first R = 2 F elements by angles p * f_i, i < F: the pairs
            (y_i, y_{i+F}), or interleaved (y_{2i}, y_{2i+1}), become
            m (a cos - b sin), m (a sin + b cos); the rest stays
  attention token j of request b, of n new tokens in a context of L, stands at
            position p = L - n + j and sees the keys c <= p with, where there
            is a window, c > p - window or c < sink
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6

# ------------------------------------------------------------------- the cases

# 64 query heads, D = 128, 64-token pages, 64 requests with contexts
# log-uniform in [4096, 131072]: the paged decode workload of this package's
# benchmark.  Its index queries: 64 heads of 128, one key for all of them.


def listed():
    return [
        # the queries and keys of one decode step: 64 requests of one token
        dict(name="rope_step", op="rope", T=64, Hq=64, Hkv=8, D=128, R=128, norm=True,
             interleaved=False, base=1e6, yarn=1.0, far=131072),
        # a whole prompt's
        dict(name="rope_prompt", op="rope", T=16384, Hq=64, Hkv=8, D=128, R=128, norm=True,
             interleaved=False, base=1e6, yarn=1.0, far=16384),
        # index queries and their shared key: half of the head rotated, in
        # neighbouring pairs, with frequencies stretched for long contexts
        dict(name="rope_index", op="rope", T=8191, Hq=64, Hkv=1, D=128, R=64, norm=False,
             interleaved=True, base=1e4, yarn=40.0, far=163840),
        # one decode step: 64 requests of two tokens, queries included
        dict(name="append_step", op="append", T=128, Hq=64, Hkv=8, D=128, R=128, norm=True,
             interleaved=False, base=1e6, yarn=1.0, far=131072, block=64, queries=True),
        # a whole prompt's keys and values
        dict(name="append_prompt", op="append", T=32768, Hq=64, Hkv=8, D=128, R=128, norm=False,
             interleaved=False, base=1e6, yarn=1.0, far=32768, block=64, queries=False),
        # a few drafted tokens of one request: what one call costs at least
        dict(name="attend_one_short", op="attend", B=1, qlo=5, qhi=5, plo=772, phi=772, Hq=64,
             Hkv=8, D=128, block=64, window=0, sink=0),
        # one token of one request with a long context: one long axis to split
        dict(name="attend_one_long", op="attend", B=1, qlo=1, qhi=1, plo=131070, phi=131070,
             Hq=64, Hkv=8, D=128, block=64, window=0, sink=0),
        # a decode batch
        dict(name="attend_decode", op="attend", B=64, qlo=1, qhi=1, plo=4095, phi=131071, Hq=64,
             Hkv=8, D=128, block=64, window=0, sink=0),
        # a prompt from its start
        dict(name="attend_prompt", op="attend", B=1, qlo=8192, qhi=8192, plo=0, phi=0, Hq=64,
             Hkv=8, D=128, block=64, window=0, sink=0),
        # a chunk of a long prompt: the largest
        dict(name="attend_chunk", op="attend", B=1, qlo=2048, qhi=2048, plo=63488, phi=63488,
             Hq=64, Hkv=8, D=128, block=64, window=0, sink=0),
        # single tokens and chunks in one batch, as requests come and go
        dict(name="attend_mixed", op="attend", B=24, qlo=1, qhi=1024, plo=100, phi=32768, Hq=16,
             Hkv=16, D=64, block=16, window=0, sink=0),
        # chunks that see a window and a few first tokens
        dict(name="attend_window", op="attend", B=8, qlo=500, qhi=2000, plo=1000, phi=65536,
             Hq=40, Hkv=8, D=128, block=32, window=4096, sink=4),
    ]


def _logu(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


MOST_PAIRS = 4 * 2048 * 64512 * 64 * 128                   # flops of attend_chunk, about
MOST_KEYS = 1 << 24                                        # keys times heads a draw's cache holds


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "attend"])
    D = rng.choice([64, 128, 128])
    Hkv = _logu(rng, 1, 16)
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 12, 16])
    if rng.random() < 0.1:
        Hkv, G = 1, rng.choice([32, 64])
    if Hkv * G > 64:
        Hkv = max(1, 64 // G)
    block = rng.choice([8, 16, 32, 64, 128])
    if op != "attend":
        far = _logu(rng, 64, 1 << 20)
        return dict(op=op, T=_logu(rng, 1, 16384 if op == "rope" else 32768), Hq=Hkv * G,
                    Hkv=Hkv, D=D, R=rng.choice([D, D, D // 2, D // 4]), norm=rng.random() < 0.5,
                    interleaved=rng.random() < 0.4, base=rng.choice([1e4, 5e5, 1e6]),
                    yarn=rng.choice([1.0, 1.0, 4.0, 40.0]), far=far,
                    **(dict(block=block, queries=rng.random() < 0.5) if op == "append" else {}))
    B = _logu(rng, 1, 64)
    phi = _logu(rng, 64, 131072)
    plo = rng.choice([0, _logu(rng, 1, phi)])
    qhi = rng.choice([1, _logu(rng, 1, 16), _logu(rng, 16, 8192)])
    qlo = _logu(rng, 1, qhi)
    window = rng.choice([0, 0, _logu(rng, 1, 8192)])
    case = dict(op=op, B=B, qlo=qlo, qhi=qhi, plo=plo, phi=phi, Hq=Hkv * G, Hkv=Hkv, D=D,
                block=block, window=window, sink=rng.choice([0, 4, 130]) if window else 0)
    while work(case)["flops"] > MOST_PAIRS // 4 or \
            sum(L for _, L in _requests(case)) * Hkv > MOST_KEYS or \
            sum(n for n, _ in _requests(case)) > 32768:
        case["phi"] = max(case["phi"] * 3 // 4, 1)
        case["plo"] = min(case["plo"], case["phi"])
        case["qhi"] = max(case["qhi"] * 3 // 4, 1)
        case["qlo"] = min(case["qlo"], case["qhi"])
        case["B"] = max(case["B"] * 7 // 8, 1)
    return case


def _spread(n, lo, hi):
    """n whole numbers spread evenly over the logarithm of [lo, hi]."""
    return [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** ((i + 0.5) / n))) - 1
            for i in range(n)]


def _requests(case):
    """(new tokens, context length) of every request."""
    B = case["B"]
    new = _spread(B, case["qlo"], case["qhi"])
    past = _spread(B, case["plo"], case["phi"])
    return [(n, n + past[(i + B // 2) % B]) for i, n in enumerate(new)]


def _seen(n, L, window, sink):
    """Pairs of a new token and a key that it sees, and keys that any sees."""
    past = L - n
    if not window or window >= L:
        return n * past + n * (n + 1) // 2, L
    pairs = 0
    for p in range(past, L):
        first = max(p - window + 1, 0)
        pairs += p + 1 - first + min(sink, first)
    first = max(past - window + 1, 0)
    return pairs, L - first + min(sink, first)


def work(case):
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    if case["op"] == "rope":
        rows = case["T"] * (Hq + Hkv)
        return dict(bytes=4 * rows * D + 4 * case["T"] + 4 * case["R"] + 8 * D * case["norm"],
                    flops=rows * (3 * case["R"] + 4 * D * case["norm"]))
    if case["op"] == "append":
        rows = case["T"] * (Hkv + Hq * case["queries"])
        return dict(bytes=4 * (rows + case["T"] * Hkv) * D + 12 * case["T"] + 4 * case["R"]
                    + 4 * D * case["norm"] * (1 + case["queries"]),
                    flops=rows * (3 * case["R"] + 4 * D * case["norm"]))
    seen = [_seen(n, L, case["window"], case["sink"]) for n, L in _requests(case)]
    tokens = sum(n for n, _ in _requests(case))
    return dict(bytes=4 * D * Hkv * sum(k for _, k in seen) + tokens * Hq * (4 * D + 4),
                flops=4 * D * Hq * sum(p for p, _ in seen))


# ---------------------------------------------------------------------- inputs


def _frequencies(case):
    """Angles per position, in 64 bits, and the factor on the rotated elements:
    base^(-2i/R); with yarn > 1, those that turn less than once in a context of
    4096 divided by it, those that turn more than 32 times kept, the others
    between by a ramp."""
    R, base, factor = case["R"], case["base"], case["yarn"]
    freq = base ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    if factor == 1.0:
        return freq, 1.0
    at = [R * math.log(4096 / (2 * math.pi * turns)) / (2 * math.log(base)) for turns in (32, 1)]
    lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), R - 1)
    ramp = ((torch.arange(R // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return freq * (1 - ramp) + freq / factor * ramp, 0.1 * math.log(factor) + 1


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _normal(g, *shape, scale=1.0):
    """Normal bf16 values, made in parts."""
    x = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    flat = x.view(-1)
    for at in range(0, flat.numel(), 1 << 28):
        part = flat[at:at + (1 << 28)]
        part.copy_(scale * _randn(g, part.numel()))
    return x


def prepare(case, seed):
    g = _gen(seed)
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    s = dict(case)
    if own:
        from top_selection_dsa_gb300 import api
        s["api"] = api
    if case["op"] != "attend":
        T = case["T"]
        # queries, keys and values as one projection writes them, token by token
        qkv = _randn(g, T, Hq + 2 * Hkv, D) * torch.exp2(_randn(g, T, Hq + 2 * Hkv, 1))
        qkv = qkv.bfloat16()
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        first = torch.randint(0, max(case["far"] - T, 0) + 1, (1,), generator=g, device=DEV)
        s["positions"] = (first + torch.arange(T, device=DEV)).int()
        s["freq"], s["factor"] = _frequencies(case)
        s["freq_dev"] = s["freq"].to(DEV)
        s["qw"] = torch.exp2(0.3 * _randn(g, D)) if case["norm"] else None
        s["kw"] = torch.exp2(0.3 * _randn(g, D)) if case["norm"] else None
        if case["op"] == "append":
            block = case["block"]
            nblk = -(-T // block) * 2
            s["slots"] = torch.randperm(nblk * block, generator=g, device=DEV)[:T].contiguous()
            s["kc"] = torch.zeros(nblk, Hkv, block, D, dtype=torch.bfloat16, device=DEV)
            s["vc"] = torch.zeros_like(s["kc"])
        if own:
            s["turns"] = s["api"].rope_turns(s["freq"])
        return s
    reqs = _requests(case)
    order = torch.randperm(len(reqs), generator=torch.Generator().manual_seed(seed)).tolist()
    reqs = s["reqs"] = [reqs[i] for i in order]
    block = case["block"]
    pages = [-(-L // block) for _, L in reqs]
    perm = torch.randperm(sum(pages), generator=g, device=DEV, dtype=torch.int32)
    s["table"] = torch.zeros(len(reqs), max(pages), dtype=torch.int32, device=DEV)
    at, starts = 0, [0]
    for b, c in enumerate(pages):
        s["table"][b, :c] = perm[at:at + c]
        at += c
        starts.append(starts[-1] + reqs[b][0])
    s["starts_host"] = starts
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    s["lens"] = torch.tensor([L for _, L in reqs], dtype=torch.int32, device=DEV)
    s["kc"] = _normal(g, at, Hkv, block, D, scale=1.5)
    s["vc"] = _normal(g, at, Hkv, block, D)
    s["q"] = _normal(g, starts[-1], Hq, D, scale=1.5)
    if own:
        s["ws"] = torch.empty(max(s["api"].kv_attention_workspace_bytes(
            starts[-1], Hq, Hkv, D), 256), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------- one pass


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    api = s["api"]
    if s["op"] == "attend":
        out, lse = api.kv_attention(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["starts"],
                                    window=s["window"], sink=s["sink"], workspace=s["ws"])
        return dict(out=out, lse=lse)
    opts = dict(k_weight=s["kw"], eps=EPS, interleaved=s["interleaved"], rope_scale=s["factor"])
    if s["op"] == "rope":
        q, k = api.qk_norm_rope(s["q"], s["k"], s["positions"], s["turns"], q_weight=s["qw"],
                                **opts)
        return dict(q=q, k=k)
    if s["queries"]:
        opts.update(q=s["q"], q_weight=s["qw"])
    kc, vc, q = api.kv_append(s["k"], s["v"], s["slots"], s["kc"], s["vc"],
                              positions=s["positions"], turns=s["turns"], **opts)
    return dict(kc=kc, vc=vc, q=q) if s["queries"] else dict(kc=kc, vc=vc)


def _norm_rope(x, weight, s):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    angle = (s["positions"].double()[:, None] * s["freq_dev"])[:, None]
    cos = (angle.cos() * s["factor"]).float()
    sin = (angle.sin() * s["factor"]).float()
    R = s["R"]
    if s["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, x[..., R:]], -1).bfloat16()


def _run_plain(s):
    if s["op"] == "rope":
        return dict(q=_norm_rope(s["q"], s["qw"], s), k=_norm_rope(s["k"], s["kw"], s))
    if s["op"] == "append":
        block = s["block"]
        page, at = s["slots"] // block, s["slots"] % block
        s["kc"][page, :, at] = _norm_rope(s["k"], s["kw"], s)
        s["vc"][page, :, at] = s["v"]
        res = dict(kc=s["kc"], vc=s["vc"])
        if s["queries"]:
            res["q"] = _norm_rope(s["q"], s["qw"], s)
        return res
    return _attend_plain(s)


def _attend_plain(s):
    D, Hq, Hkv, block = s["D"], s["Hq"], s["Hkv"], s["block"]
    G = Hq // Hkv
    out = torch.empty_like(s["q"])
    lse = torch.empty(s["q"].shape[:2], device=DEV)
    for b, (n, L) in enumerate(s["reqs"]):
        rows = slice(s["starts_host"][b], s["starts_host"][b] + n)
        pages = s["table"][b, :-(-L // block)].long()
        p = torch.arange(L - n, L, device=DEV)[:, None]
        first = max(L - n - s["window"] + 1, 0) if s["window"] else 0
        c = torch.arange(L, device=DEV)
        if first > s["sink"]:                              # nothing sees the keys between
            c = torch.cat([c[:s["sink"]], c[first:]])
        hidden = c > p
        if s["window"]:
            hidden = hidden | ((c <= p - s["window"]) & (c >= s["sink"]))
        page, at = pages[c // block], c % block
        heads = max(1, min(Hkv, (1 << 31) // (n * G * c.numel())))
        for h in range(0, Hkv, heads):
            K = s["kc"][page, h:h + heads, at].float()     # [keys, heads, D]
            V = s["vc"][page, h:h + heads, at].float()
            m = K.shape[1]
            q = s["q"][rows, h * G:(h + m) * G].float().reshape(n, m, G, D)
            q = q.permute(1, 2, 0, 3).reshape(m, G * n, D)
            S = torch.matmul(q, K.permute(1, 2, 0)) * D ** -0.5
            S = S.view(m, G, n, -1).masked_fill_(hidden, -torch.inf)
            top = S.amax(-1, keepdim=True)
            S = S.sub_(top).exp_()
            l = S.sum(-1, keepdim=True)
            o = torch.matmul(S.view(m, G * n, -1), V.transpose(0, 1)).view(m, G, n, D) / l
            out[rows, h * G:(h + m) * G] = o.permute(2, 0, 1, 3).reshape(n, m * G, D).bfloat16()
            lse[rows, h * G:(h + m) * G] = (top + l.log())[..., 0].permute(2, 0, 1).reshape(n, -1)
    return dict(out=out, lse=lse)


# ------------------------------------------------------------------ definitions


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "rope":
        return dict(q=_turn64(s["q"], s["qw"], s), k=_turn64(s["k"], s["kw"], s))
    if case["op"] == "append":
        k, v = _turn64(s["k"], s["kw"], s), s["v"].double()
        kc, vc = s["kc"].double(), s["vc"].double()
        block = case["block"]
        for h in range(case["Hkv"]):
            kc[:, h] = kc[:, h].reshape(-1, case["D"]).index_copy(0, s["slots"], k[:, h]) \
                .view(-1, block, case["D"])
            vc[:, h] = vc[:, h].reshape(-1, case["D"]).index_copy(0, s["slots"], v[:, h]) \
                .view(-1, block, case["D"])
        res = dict(kc=kc, vc=vc)
        if case["queries"]:
            res["q"] = _turn64(s["q"], s["qw"], s)
        return res
    if work(case)["flops"] > 3 << 40:
        return None
    return _attend64(s)


def _turn64(x, weight, s):
    """Pairs as complex numbers times m e^(i angle), in 64 bits."""
    x = x.double()
    if weight is not None:
        x = x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * weight.double()
    angle = s["positions"].double()[:, None, None] * s["freq_dev"]
    turn = torch.polar(torch.full_like(angle, s["factor"]), angle)
    R, F = s["R"], s["R"] // 2
    i = torch.arange(F, device=DEV)
    ia, ib = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + F)
    y = x.clone()
    z = torch.complex(x[..., ia], x[..., ib]) * turn
    y[..., ia], y[..., ib] = z.real, z.imag
    assert R <= x.shape[-1]
    return y


def _attend64(s):
    D, Hq, Hkv, block = s["D"], s["Hq"], s["Hkv"], s["block"]
    G = Hq // Hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    for b, (n, L) in enumerate(s["reqs"]):
        t0 = s["starts_host"][b]
        for h in range(Hkv):
            pages = s["table"][b].long()[:-(-L // block)]
            K = s["kc"][pages, h].reshape(-1, D)[:L].double()
            V = s["vc"][pages, h].reshape(-1, D)[:L].double()
            step = max(1, (1 << 27) // (L * G))
            for j in range(0, n, step):
                m = min(step, n - j)
                p = torch.arange(L - n + j, L - n + j + m, device=DEV)
                lo, hi = 0, L - n + j + m
                if s["window"] and s["sink"] == 0:
                    lo = max(0, L - n + j - s["window"] + 1)
                c = torch.arange(lo, hi, device=DEV)
                sees = c[None] <= p[:, None]
                if s["window"]:
                    sees &= (p[:, None] - c[None] < s["window"]) | (c[None] < s["sink"])
                q = s["q"][t0 + j:t0 + j + m, h * G:(h + 1) * G].double()
                S = torch.einsum("tgd,cd->tgc", q, K[lo:hi]) / math.sqrt(D)
                S = torch.where(sees[:, None], S, -math.inf)
                z = torch.logsumexp(S, -1)
                lse[t0 + j:t0 + j + m, h * G:(h + 1) * G] = z
                out[t0 + j:t0 + j + m, h * G:(h + 1) * G] = \
                    torch.einsum("tgc,cd->tgd", torch.exp(S - z[..., None]), V[lo:hi])
    return dict(out=out, lse=lse)
