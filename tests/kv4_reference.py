"""Plain 64-bit implementations of the 4-bit key/value cache operators, written
from the definitions in include/dsa.h; numpy on the CPU."""
import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def encode(x):
    """[..., D] float64 -> (codes [..., D] uint8, scales [..., D/32] uint8)."""
    lead, D = x.shape[:-1], x.shape[-1]
    blk = x.reshape(*lead, D // 32, 32)
    codes = np.zeros(blk.shape, np.uint8)
    scales = np.zeros(blk.shape[:-1], np.uint8)
    for i in np.ndindex(*blk.shape[:-1]):
        v = blk[i]
        if not np.isfinite(v).all():
            scales[i] = 255
            continue
        amax = np.abs(v).max()
        e = 0
        if amax > 0:
            e = -126
            while amax > 6 * 2.0 ** e:
                e += 1
        scales[i] = e + 127
        for j, a in enumerate(np.abs(v) / 2.0 ** e):
            d = np.abs(E2M1[:8] - a)
            best = min(range(8), key=lambda c: (d[c], c & 1))
            codes[i][j] = best | (8 if np.signbit(v[j]) else 0)
    return codes.reshape(*lead, D), scales


def _byte_of(D, e, value):
    """(byte, nibble) of element e of a record's key (value) half."""
    G = D // 32
    g = e // 32
    if value:
        return D // 2 + ((e % 32 // 4) * G + g) * 2 + e % 4 // 2, e % 2
    return ((e % 32 // 8) * G + g) * 4 + e % 8 // 2, e % 2


def pack(kc, vc):
    """Codes [..., D] of key and value -> records [..., D]."""
    D = kc.shape[-1]
    rec = np.zeros(kc.shape, np.uint8)
    for c, value in ((kc, False), (vc, True)):
        for e in range(D):
            byte, nib = _byte_of(D, e, value)
            rec[..., byte] |= c[..., e] << (4 * nib)
    return rec


def decode(rec, sc):
    """Records and scales [..., D], [..., D/16] -> key and value [..., D] float64."""
    D = rec.shape[-1]
    G = D // 32
    out = []
    for value in (False, True):
        x = np.zeros(rec.shape)
        s = sc[..., G:] if value else sc[..., :G]
        f = np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(int) - 127))
        for e in range(D):
            byte, nib = _byte_of(D, e, value)
            x[..., e] = E2M1[(rec[..., byte] >> (4 * nib)) & 15] * f[..., e // 32]
        out.append(x)
    return out


def attention(q, K, V, scale, seen, cols=None):
    """One row's heads: q [Hq, D], K/V [L, Hkv, D]; columns `cols` (default
    all) below `seen`.  Returns (out, lse, weights per entry of cols, bound):
    bound holds, per head, sum p|V| [D], and the largest sum |q||k| scale."""
    Hq, D = q.shape
    Hkv = K.shape[1]
    G = Hq // Hkv
    cols = np.arange(K.shape[0]) if cols is None else cols
    out, lse = np.zeros((Hq, D)), np.full(Hq, -np.inf)
    A, Bd = np.zeros((Hq, D)), np.zeros(Hq)
    w = np.zeros(len(cols))
    ok = (cols >= 0) & (cols < seen)
    c = cols[ok]
    if len(c):
        for h in range(Hq):
            k, v = K[c, h // G], V[c, h // G]
            S = scale * (k @ q[h])
            m = S.max()
            p = np.exp(S - m)
            l = p.sum()
            lse[h] = m + np.log(l)
            p = p / l
            out[h] = p @ v
            A[h] = p @ np.abs(v)
            Bd[h] = abs(scale) * (np.abs(k) @ np.abs(q[h])).max()
            w[ok] += p
    return out, lse, w, (A, Bd)


def evict(w, L, budget, sink, recent):
    lo = min(sink, L)
    hi = max(lo, L - recent)
    mid = [i for i in range(lo, hi) if np.isfinite(w[i]) or w[i] == np.inf]
    mid = sorted(mid, key=lambda i: (-w[i], i))[:budget - sink - recent]
    return sorted(list(range(lo)) + mid + list(range(hi, L)))
