"""Single rows of attention over the 4-bit cache in 64 bits, with a bound that follows each token's own
weight, and how a call is cut (a copy of the rule in csrc/kv4_attention.hip, so that a test knows which
kernels its sizes reach)."""
import numpy as np

from attention_ref import rounding


def attention_rows(q, name, cache, table, kv_lens, cu_q, rows, scale=None, causal=True, window=0, run=None):
    """(o, lse, bound of o, bound of lse) of the rows [(token, head)] of q [T, Hq, D], numbers of type `name`.

    run: the most tokens that one wave adds up (all that a row sees when None).  With P_j = p_j s_j, c_j the
    value's code and `largest` the row's largest P_j, the bound counts
      - `wrong`: a score's sum has D / 8 + 4 additions of fp32 (twice that is allowed) of up to 16 |q|, products
        cut below 2^-18 of the largest |q|, numbers held in fp16 with 2^-25 of 1, or of what its row is
        brought to; an exponent of size e is off by 4 e 2^-24, exp2, log2 and reciprocal by 16 2^-24.  It
        moves P_j c_j in the numerator and p_j in the sum by that much of themselves;
      - a weight is rounded to fp16: 2^-11 of itself, or half fp16's smallest step where the row's largest
        weight is at least 2^7, so 2^-32 of `largest`;
      - products of 32 tokens, with the code (up to 15) and with the offset of 8, cut below 2^-18 of their
        largest weight each, and by no more than there is of them;
      - run / 8 + 64 additions of fp32 to the sums of P_j (c_j + 8) and 8 P_j, run / 4 + 64 to the row's.
    """
    T, Hq, D = q.shape
    share = Hq // cache.kc.shape[1]
    scale = D ** -0.5 if scale is None else scale
    cu_q = np.arange(len(table) + 1) if cu_q is None else np.asarray(cu_q)
    o, lse, bound, lse_bound = np.zeros((len(rows), D)), np.zeros(len(rows)), np.zeros((len(rows), D)), np.zeros(len(rows))
    for at, (t, h) in enumerate(rows):
        b = int(np.searchsorted(cu_q[1:], t, side="right"))
        i, n, kv, g = t - int(cu_q[b]), int(cu_q[b + 1] - cu_q[b]), int(kv_lens[b]), h // share
        hi = kv - n + i + 1 if causal else kv
        j = np.arange(max(0, hi - window) if window else 0, hi)
        pages = table[b, j // cache.page]
        j = j[(pages >= 0) & (pages < len(cache.kc))]
        lse[at] = -np.inf
        if len(j) == 0:
            continue
        p, off = table[b, j // cache.page], j % cache.page
        x = np.asarray(q[t, h], np.float64)
        ks, vs = cache.ks[p, g, off].astype(np.float64), cache.vs[p, g, off].astype(np.float64)
        c = cache.vc[p, g, off].astype(np.float64)
        s = scale * (cache.kc[p, g, off] @ x) * ks
        w = np.exp(s - s.max())
        total = w.sum()
        P, pr = w * vs / total, w / total
        o[at] = P @ c
        lse[at] = s.max() + np.log(total)
        most, many = np.abs(x).max(), len(j) if run is None else min(run, len(j))
        level = 1.0 if 2.0 ** -6 <= most < 2.0 ** 14 else most * 2.0 ** -4
        held = 16 * D * 2.0 ** -25 * level + 2 * D * 2.0 ** -18 * most \
            + (D / 4 + 8) * 2.0 ** -24 * 16 * np.abs(x).sum()
        e = 1.45 * np.abs(s) + np.abs(np.log2(np.maximum(vs, 2.0 ** -80)))
        wrong = scale * held * ks + (4 * e + 16) * 2.0 ** -24
        largest = P.max()
        chunks = np.zeros(int(j[-1]) // 32 + 1)
        np.maximum.at(chunks, j // 32, P)
        dropped = np.minimum(23 * P, 2 * 2.0 ** -18 * chunks[j // 32]).sum()
        sizes = np.abs(c)
        bound[at] = (wrong * P) @ sizes + np.abs(o[at]) * (wrong @ pr) \
            + np.maximum(2.0 ** -11 * P, 2.0 ** -32 * largest) @ sizes + dropped \
            + (many / 8 + 64) * 2.0 ** -24 * (P @ (c + 16)) + (many / 4 + 64) * 2.0 ** -24 * np.abs(o[at]) \
            + 8 * 2.0 ** -80 + rounding(o[at], name)
        lse_bound[at] = wrong.max() + (many / 4 + 64) * 2.0 ** -24 + np.abs(lse[at]) * 2.0 ** -22
    return o, lse, bound, lse_bound


def cut(T, B, Hq, Hkv, D, max_q, max_kv, window=0, cus=256):
    """How kv4_attention cuts a call: "rows" or "few", the row tiles of 16 a wave, whether the batch is
    numbered unevenly, tiles shared by several workgroups (and in many parts), the longest first."""
    share, pairs = Hq // Hkv, B * Hkv
    max_q = max(1, min(max(max_q, -(-T // B)), T))
    each, wide = max_q * share, 2 ** 24 - 1
    rt = 1 if D == 256 or each <= 16 else 2

    def tile(R):
        n, places = -(-each // R), (T * share // R + B) * Hkv
        uneven = places < pairs * n and places <= wide
        return (0 if uneven else max(1, min(n, wide // pairs))), places

    def blocks(tiles, places):
        return pairs * tiles if tiles else places
    tiles, places = tile(64 * rt)
    if each > 16 * rt and 2 * blocks(tiles, places) >= 3 * cus:
        return dict(kernel="rows", rt=rt, uneven=tiles == 0, share=False, deep=False, sorted=False)
    tiles, places = tile(16 * rt)
    n = blocks(tiles, places)
    seen = min(max_kv, window + 16 * rt // share) if window else max_kv
    units = -(-seen // 256)
    split = units > 5 and n < 2 * cus
    return dict(kernel="few", rt=rt, uneven=tiles == 0, share=split,
                deep=split and units * min(n * units, 2 * cus) > 8 * n * units,
                sorted=not split and tiles > 0 and units > 5 and 1 < B <= 256)
