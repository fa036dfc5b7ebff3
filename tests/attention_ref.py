"""Plain implementations in 64 bits of rotary positions, the 4-bit key/value cache and attention
over it (include/apex4.h), with the bounds that a right computation keeps to."""
import numpy as np

EPS = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}      # half a step, relative
TINY = {"float32": 2.0 ** -150, "float16": 2.0 ** -25, "bfloat16": 2.0 ** -134}  # half the smallest step


def rounding(x, name):
    """How far rounding to a type may move the numbers x."""
    return np.abs(x) * EPS[name] + TINY[name]


def off(got, want, bound, name):
    """Where got is further from want than bound.  A number that may reach the middle between the
    type's largest and the power of two above it (fp16: 65504 and 65536) rounds to infinity."""
    most = {"float32": 2.0 ** 128, "float16": 65520.0, "bfloat16": 2.0 ** 128 - 2.0 ** 119}[name]
    over = np.isinf(got) & (np.sign(got) == np.sign(want)) & (np.abs(want) + bound >= most)
    with np.errstate(invalid="ignore"):
        return ~(np.abs(got - want) <= bound) & ~over


# ---------------------------------------------------------------- rotary positions

def frequencies(R, base=10000.0, stretch=1.0):
    return base ** (-np.arange(R // 2, dtype=np.float64) / (R // 2)) / stretch


def rope(x, positions, freqs, interleaved=False, scale=1.0):
    """x [T, H, D] in float64 -> the turned numbers, unrounded."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    R = 2 * len(freqs)
    for t, p in enumerate(positions):
        theta = np.float64(p) * freqs
        c, s = scale * np.cos(theta), scale * np.sin(theta)
        a = x[t, :, 0:R:2] if interleaved else x[t, :, :R // 2]
        b = x[t, :, 1:R:2] if interleaved else x[t, :, R // 2:R]
        first, second = a * c - b * s, b * c + a * s
        if interleaved:
            y[t, :, 0:R:2], y[t, :, 1:R:2] = first, second
        else:
            y[t, :, :R // 2], y[t, :, R // 2:R] = first, second
    return y


# ---------------------------------------------------------------- the cache

def codes(x):
    """(codes -8..7, scales) of the heads x [..., D], fp32 numbers, by the quantization rule."""
    x = np.asarray(x, np.float32)
    a = np.abs(x).max(-1)
    finite = np.isfinite(x).all(-1)
    s = np.where(finite, np.where(finite, a, 0) / np.float32(7), np.float32(np.nan)).astype(np.float32)
    c = np.zeros(x.shape, np.int64)
    live = finite & (s > 0)
    c[live] = np.clip(np.rint(x[live] / s[live][..., None]), -8, 7).astype(np.int64)
    return c, s


class Cache:
    """A cache on the host: codes [pages, heads, page, D] and scales of keys and values."""

    def __init__(self, pages, heads, page, D, seed=0):
        rng = np.random.default_rng(seed)
        shape = (pages, heads, page)
        self.page, self.D = page, D
        self.kc, self.vc = (rng.integers(-8, 8, shape + (D,)) for _ in range(2))
        self.ks = rng.uniform(0.05, 0.4, shape).astype(np.float32)
        self.vs = rng.uniform(0.05, 0.4, shape).astype(np.float32)

    @staticmethod
    def value_places(page, D):
        """(row, byte, shift) of every (token, number) of a page's values."""
        off, d = np.arange(page)[:, None], np.arange(D)[None, :]
        byte = (16 * (off % 16 // 4) + d % 16) * (D // 8) + 4 * (d // 32) + off % 4
        return off // 16 + 0 * d, byte, np.where(d % 32 >= 16, 4, 0) + 0 * off

    def arrays(self):
        """(k_codes, k_scales, v_codes, v_scales) as the library keeps them."""
        pages, heads, page, D = self.kc.shape
        k = (self.kc + 8).astype(np.uint8)
        v = np.zeros((pages, heads, page // 16, 8 * D), np.uint8)
        row, byte, shift = self.value_places(page, D)
        for half in (0, 4):
            at = shift == half
            v[:, :, row[at], byte[at]] |= ((self.vc[:, :, at] + 8) << half).astype(np.uint8)
        return k[..., 0::2] | (k[..., 1::2] << 4), self.ks, v, self.vs

    @classmethod
    def of(cls, k_codes, k_scales, v_codes, v_scales):
        c = cls.__new__(cls)
        pages, heads, page, half = k_codes.shape
        c.page, c.D = page, 2 * half
        c.kc = np.stack((k_codes & 15, k_codes >> 4), -1).reshape(pages, heads, page, -1).astype(np.int64) - 8
        row, byte, shift = cls.value_places(page, c.D)
        c.vc = ((v_codes[:, :, row, byte] >> shift) & 15).astype(np.int64) - 8
        c.ks, c.vs = k_scales.copy(), v_scales.copy()
        return c

    def put(self, slots, k, v):
        """Stores tokens' fp32 keys and values [T, heads, D]; slots outside the cache are not stored."""
        (kc, ks), (vc, vs) = codes(k), codes(v)
        for t, slot in enumerate(slots):
            p, off = divmod(int(slot), self.page)
            if 0 <= p < len(self.kc):
                self.kc[p, :, off], self.ks[p, :, off] = kc[t], ks[t]
                self.vc[p, :, off], self.vs[p, :, off] = vc[t], vs[t]

    def values(self, slots):
        """(keys, values) [T, heads, D] in float64."""
        slots = np.asarray(slots, np.int64)
        live = (slots >= 0) & (slots // self.page < len(self.kc))
        p, off = np.where(live, slots // self.page, 0), np.where(live, slots % self.page, 0)
        out = []
        for c, s in ((self.kc, self.ks), (self.vc, self.vs)):
            x = c[p, :, off] * s[p, :, off].astype(np.float64)[..., None]
            out.append(np.where(live[:, None, None], x, 0.0))
        return out


# ---------------------------------------------------------------- attention

def attention(q, name, cache, table, kv_lens, cu_q, scale=None, causal=True, window=0):
    """(o, lse, bound of o, bound of lse, owned rows) of q [T, Hq, D], numbers of type `name`.

    The bound counts, for a row that sees n tokens, every rounding that the
    header allows:
      - a query is held in fp16 beside codes up to 15: 2^-25 of its row's scale a
        number at the least, where that scale is 1 for rows whose largest number is
        between 2^-6 and 2^14, and brings the others there;
      - D products, and the offset of 8 in every code, sum in fp32: 2 D 2^-24 of
        sum |q| 16 s_k; and each is cut below 2^-18 of its eight's largest |q|;
      - an exponent of size e is off by 4 e 2^-24, exp2, log2 and reciprocal by
        4 units of fp32: together `wrong`, which moves every p_j by that much of
        itself, twice (numerator and sum);
      - p_j s_j is rounded to fp16, relative to 2^-11, or 2^-25 of the largest, and
        its product with a code, and with the offset, cut below 2^-18 of that;
      - n / 32 sums of products of weights and codes up to 15, in fp32.
    """
    q = np.asarray(q, np.float64)
    T, Hq, D = q.shape
    heads = cache.kc.shape[1]
    share = Hq // heads
    scale = D ** -0.5 if scale is None else scale
    B, cols = table.shape
    o, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    bound, lse_bound = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    owned = np.zeros(T, bool)
    cu_q = np.arange(B + 1) if cu_q is None else np.clip(cu_q, 0, T)
    for b in range(B):
        start, n = int(cu_q[b]), int(cu_q[b + 1] - cu_q[b])
        owned[start:start + n] = True
        kv = min(max(int(kv_lens[b]), 0), cols * cache.page)
        if kv == 0 or n <= 0:
            continue
        j = np.arange(kv)
        pages = table[b, j // cache.page].astype(np.int64)
        live = (pages >= 0) & (pages < len(cache.kc))
        slots = np.where(live, pages * cache.page + j % cache.page, -1)
        p, off = np.where(live, pages, 0), j % cache.page
        pos = kv - n + np.arange(n)[:, None]
        seen = live[None] & ((j <= pos) & ((j > pos - window) | (window == 0)) if causal else j < kv)
        with np.errstate(invalid="ignore", over="ignore"):
            keys, vals = cache.values(slots)
            for h in range(Hq):
                g = h // share
                x = q[start:start + n, h]
                ks, vs = cache.ks[p, g, off].astype(np.float64), cache.vs[p, g, off].astype(np.float64)
                t = np.where(seen, scale * (x @ keys[:, g].T), -np.inf)
                some = seen.any(-1)
                top = np.where(some, t.max(-1), 0.0)
                w = np.where(seen, np.exp(t - top[:, None]), 0.0)
                total = w.sum(-1)
                pr = w / np.where(some, total, 1.0)[:, None]
                v = np.where(live[:, None], vals[:, g], 0.0)
                gone = ~seen.any(0)                        # (what nobody sees may hold NaN)
                v[gone] = 0.0
                vs = np.where(gone, 0.0, vs)
                ks = np.where(gone, 0.0, ks)
                r = np.where(some[:, None], pr @ v, 0.0) if np.isfinite(v).all() else \
                    np.stack([(pr[i][seen[i]] @ v[seen[i]]) if some[i] else np.zeros(D) for i in range(n)])
                o[start:start + n, h] = r
                lse[start:start + n, h] = np.where(some, top + np.log(np.where(some, total, 1.0)), -np.inf)
                most = np.abs(x).max(-1)
                level = np.where((most >= 2.0 ** -6) & (most < 2.0 ** 14), 1.0, most * 2.0 ** -4)
                held = 16 * D * 2.0 ** -25 * level + 2 * D * 2.0 ** -18 * most \
                    + 2 * D * 2.0 ** -24 * 16 * np.abs(x).sum(-1)
                with np.errstate(divide="ignore"):
                    e = np.abs(np.where(seen, t, 0.0)) * 1.45 + np.abs(np.log2(np.maximum(vs, 2.0 ** -80)))
                wrong = (scale * held[:, None] * np.where(seen, ks, 0.0) + (4 * e + 16) * 2.0 ** -24).max(-1)
                ps = pr * np.where(seen, vs, 0.0)
                count = seen.sum(-1)
                each = 8 * ps.sum(-1) * (2 * wrong + 2.0 ** -11) + count * (8 * 2.0 ** -25 + 2 * 2.0 ** -18) * ps.max(-1) \
                    + 15 * ps.sum(-1) * (count / 16 + 64) * 2.0 ** -24 + 15 * 2.0 ** -60
                bound[start:start + n, h] = each[:, None] + rounding(r, name)
                lse_bound[start:start + n, h] = wrong + (count / 16 + 64) * 2.0 ** -24 \
                    + np.abs(np.where(some, lse[start:start + n, h], 0)) * 2.0 ** -22
    return o, lse, bound, lse_bound, owned
