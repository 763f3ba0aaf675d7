"""Plain 64-bit restatements of the 8-bit operators (CPU, numpy), for the tests.

Written from the operators' definitions in include/vocoder.h; they share no code with the
library.  e4m3 values are handled as numbers: `e4m3_round` rounds to the format's grid."""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
BLOCK = 64


def e4m3_round(v):
    """Nearest e4m3 value (ties to even), magnitudes over 448 to 448, NaN kept."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.where(a > 0, a, 1.0)))
    e = np.where(np.ldexp(1.0, np.nan_to_num(e, posinf=0, neginf=0).astype(int)) > a, e - 1, e)
    e = np.clip(np.nan_to_num(e, posinf=8.0, neginf=-6.0), -6, 8)  # smallest normal 2^-6
    step = np.exp2(e - 3)
    r = np.minimum(np.where(np.isinf(a), E4M3_MAX, np.rint(np.where(np.isinf(a), 0, a) / step) * step),
                   E4M3_MAX)
    return np.where(np.isnan(v), np.nan, np.copysign(r, v))


def rows(x, mode, weight=None, residual=None, eps=1e-6):
    """(n, scale, h): normalised rows before rounding, scale per row, sum."""
    h = x.astype(np.float64)
    if residual is not None:
        h = h + residual.astype(np.float64)
    if mode == "rms":
        with np.errstate(invalid="ignore", divide="ignore"):
            rms = np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
            n = np.where(rms == 0, 0, h / rms) * weight.astype(np.float64)
    elif mode == "gated":
        d = h.shape[1] // 2
        with np.errstate(over="ignore"):
            n = h[:, :d] / (1 + np.exp(-h[:, :d])) * h[:, d:]
    else:
        n = h
    scale = np.maximum(np.max(np.abs(n), axis=1), 2.0 ** -96) / E4M3_MAX
    return n, scale, h


def block_scale(amax):
    """Smallest 2^e, e >= -96, with amax <= 448 * 2^e."""
    e = -96
    while amax > E4M3_MAX * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(kc, vc, ks, vs, k, v, table, lens, new):
    """The cache (codes' values [page][head][64][d], [page][head][d][64]; scales) after appending
    k, v [token][head][d]; `new` tokens of each sequence.  In place."""
    pages, heads = ks.shape
    at = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        p0 = n - m
        touched = {}
        for i in range(m):
            pos = p0 + i
            if pos >= 0 and pos // BLOCK < table.shape[1]:
                page = table[b, pos // BLOCK]
                if 0 <= page < pages:
                    touched.setdefault(page, []).append((pos % BLOCK, at + i))
        at += m
        for page, toks in touched.items():
            slots = np.array([s for s, _ in toks])
            idx = np.array([i for _, i in toks])
            fresh = slots[0] == 0
            for h in range(heads):
                nk, nv = k[idx, h].astype(np.float64), v[idx, h].astype(np.float64)  # [token][d]
                bad = np.isnan(nk).any(1) | np.isnan(nv).any(1)
                for c, s, new_v, tr in ((kc, ks, nk, False), (vc, vs, nv, True)):
                    fin = np.abs(new_v[np.isfinite(new_v)])
                    sc = block_scale(fin.max() if fin.size else 0.0)
                    blk = c[page, h].T if tr else c[page, h]  # [slot][d]
                    if fresh:
                        blk[:] = 0
                    else:
                        sc = max(sc, s[page, h])
                        if sc != s[page, h]:
                            blk[:] = e4m3_round(blk * (s[page, h] / sc))
                    q = e4m3_round(np.where(np.isnan(new_v), 0, new_v) / sc)
                    if not tr:
                        q[bad] = np.nan
                    blk[slots] = q
                    s[page, h] = sc


def attention(q, kc, vc, ks, vs, table, lens, new, scale, causal=True, window=0):
    """(o, a, s): output, sum of weights times |v| (for error bounds) and the largest sum over d of
    |q k| * scale a row meets, each for [token][head]."""
    tokens, heads, d = q.shape
    kv_heads = kc.shape[1]
    group = heads // kv_heads
    o = np.zeros((tokens, heads, d))
    a = np.zeros((tokens, heads, d))
    smax = np.zeros((tokens, heads))
    at = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        cap = min(n, table.shape[1] * BLOCK)
        for i in range(m):
            pos = n - m + i
            hi = min(cap, pos + 1) if causal else cap
            lo = max(0, pos - window + 1) if window else 0
            keys = [j for j in range(lo, max(lo, hi)) if 0 <= table[b, j // BLOCK] < len(kc)]
            if not keys:
                continue
            j = np.array(keys)
            page, slot = table[b, j // BLOCK], j % BLOCK
            for h in range(heads):
                g = h // group
                kk = kc[page, g, slot] * ks[page, g][:, None]
                vv = vc[page, g, :, slot] * vs[page, g][:, None]
                qq = q[at + i, h].astype(np.float64)
                s = kk @ qq * scale
                with np.errstate(invalid="ignore"):
                    w = np.exp(s - s.max())
                w = w / w.sum()
                o[at + i, h] = w @ vv
                a[at + i, h] = w @ np.abs(vv)
                smax[at + i, h] = np.max(np.abs(kk) @ np.abs(qq)) * abs(scale)
        at += m
    return o, a, smax
