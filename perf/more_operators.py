"""Operators between a decoder layer's projections, as cases to measure.

Four operators around a key/value cache held in 4 bits: rotary positions
("rope"), appending rotated keys and values to the paged cache ("append"),
reading cached tokens back ("read"), and attention over the cache ("attend").
With `own` false, `run` computes them from elementary torch operations; with
`own` true it calls this repository's entry points.

The cache is four tensors.  A key's or value's head of D numbers is kept as
codes c = clamp(round(x / s), -8, 7), s = max|x| / 7, each stored as the
nibble c + 8:
    k_codes  [pages, heads, page, D/2]      code d in byte d/2, even d low
    v_codes  [pages, heads, page/16, 8 D]   16 tokens at a time; token 4 g + i and the dims r + 32 v (low nibble)
                                            and r + 32 v + 16 (high), r < 16, in byte (16 g + r) D/8 + 4 v + i
    k_scales, v_scales  [pages, heads, page]
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token's queries in the 7B shape, 32 heads of 128: latency
        dict(name="rope-token", op="rope", tokens=1, heads=32, dim=128, rotary=128, interleaved=False, first=4000,
             stretch=1.0, dtype="float16"),
        # the 70B shape's 64 heads of a long prompt, far positions with stretched frequencies, half of each head
        dict(name="rope-prompt", op="rope", tokens=4096, heads=64, dim=128, rotary=64, interleaved=True,
             first=1000000, stretch=8.0, dtype="bfloat16"),
        # one decoding step of one sequence, 7B shape
        dict(name="append-token", op="append", tokens=1, heads=32, kv_heads=32, dim=128, page=16, rotary=128,
             interleaved=False, first=516, stretch=1.0, padded=0, prompt=False, dtype="float16"),
        # one decoding step of a batch with padded places, 70B shape: every token goes to a page of its own
        dict(name="append-batch", op="append", tokens=61, heads=64, kv_heads=8, dim=128, page=64, rotary=128,
             interleaved=False, first=3000, stretch=1.0, padded=5, prompt=False, dtype="bfloat16"),
        # a whole prompt, 70B shape, the rotation on neighbouring pairs of half the head
        dict(name="append-prompt", op="append", tokens=4096, heads=64, kv_heads=8, dim=128, page=64, rotary=64,
             interleaved=True, first=0, stretch=4.0, padded=0, prompt=True, dtype="float16"),
        # a short prefix copied out of the cache, 7B shape
        dict(name="read-prefix", op="read", tokens=517, kv_heads=32, dim=128, page=16, dtype="float16"),
        # a long one, 70B shape
        dict(name="read-long", op="read", tokens=65521, kv_heads=8, dim=128, page=128, dtype="bfloat16"),
        # a decoding step of one short sequence, 7B shape, no shared heads: latency
        dict(name="attend-token", op="attend", batch=1, q=1, kv=517, ragged=False, heads=32, kv_heads=32, dim=128,
             page=16, window=0, dtype="float16"),
        # a decoding step of 64 sequences of all lengths, 8 query heads to a key head
        dict(name="attend-decode", op="attend", batch=64, q=1, kv=8192, ragged=True, heads=64, kv_heads=8, dim=128,
             page=64, window=0, dtype="bfloat16"),
        # a decoding step of one very long sequence: the cache's axis has to be split
        dict(name="attend-long", op="attend", batch=1, q=1, kv=131071, ragged=False, heads=64, kv_heads=8, dim=128,
             page=128, window=0, dtype="float16"),
        # prompts taken in parts beside decoding sequences, small heads, a window
        dict(name="attend-chunks", op="attend", batch=5, q=301, kv=6011, ragged=True, heads=16, kv_heads=4, dim=64,
             page=32, window=1000, dtype="bfloat16"),
        # a whole prompt, 70B shape
        dict(name="attend-prompt", op="attend", batch=1, q=4096, kv=4096, ragged=False, heads=64, kv_heads=8, dim=128,
             page=64, window=0, dtype="float16"),
    ]


_PAIRS = 4096 * 4097 // 2 * 64 * 128          # of query and key, times heads times dims: the longest listed prompt
_CACHE = 64 * 4300 * 8 * 136                  # bytes of cache of the listed decoding batch


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "append", "append", "read", "attend", "attend", "attend", "attend"))
    dim = rng.choice((64, 128, 128, 256))
    kv_heads = rng.choice((1, 2, 4, 8, 8, 16, 32))
    heads = kv_heads * min(64 // kv_heads, rng.choice((1, 1, 2, 4, 5, 7, 8, 16)))
    page = rng.choice((16, 32, 64, 128, 256))
    dtype = rng.choice(("float16", "bfloat16"))
    turn = dict(rotary=rng.choice((dim, dim, dim // 2, dim // 4)), interleaved=rng.random() < 0.5,
                first=_log_int(rng, 1, 1 << 20) - 1, stretch=rng.choice((1.0, 1.0, 4.0, 8.0)))
    if op == "rope":
        return dict(op=op, tokens=_log_int(rng, 1, 4096 * 64 * 128 // (heads * dim)), heads=heads, dim=dim,
                    dtype=rng.choice(("float16", "bfloat16", "float32")), **turn)
    if op == "append":
        tokens = _log_int(rng, 1, min(8192, 4096 * 80 * 128 // ((heads + 2 * kv_heads) * dim)))
        return dict(op=op, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                    padded=rng.randint(0, tokens // 4), prompt=rng.random() < 0.5, dtype=dtype, **turn)
    if op == "read":
        return dict(op=op, tokens=_log_int(rng, 1, min(65521, 65521 * 8 * 128 // (kv_heads * dim))),
                    kv_heads=kv_heads, dim=dim, page=page, dtype=rng.choice(("float16", "bfloat16", "float32")))
    q = rng.choice((1, 1, _log_int(rng, 2, 64), _log_int(rng, 64, 4096)))
    batch = _log_int(rng, 1, 64) if q < 64 else rng.randint(1, 4)
    most = min(131071, _CACHE // (batch * kv_heads * (dim + 8)), max(q, _PAIRS // (batch * q * heads * dim)))
    kv = _log_int(rng, max(q, 16), max(q, 16, most))
    while batch > 1 and batch * kv * q * heads * dim > _PAIRS:
        batch -= 1
    while batch * kv * q * heads * dim > 2 * _PAIRS:
        q, kv = (q + 1) // 2, max((q + 1) // 2, kv // 2)
    return dict(op=op, batch=batch, q=q, kv=kv, ragged=batch > 1 and rng.random() < 0.75, heads=heads,
                kv_heads=kv_heads, dim=dim, page=page, window=rng.choice((0, 0, 0, _log_int(rng, 16, 4096))),
                dtype=dtype)


def _lengths(case):
    """(new tokens, cached tokens with them) of every sequence, from the case alone."""
    b, q, kv = case["batch"], case["q"], case["kv"]
    if not case["ragged"]:
        return [q] * b, [kv] * b
    rng = random.Random(1000003 * b + 1009 * q + kv)
    news, olds = [q], [kv]
    for _ in range(b - 1):
        news.append(_log_int(rng, 1, q))
        olds.append(rng.randint(news[-1], kv))
    if b > 8:
        news[-1], olds[-1] = 1, 0                          # a place of the batch that holds no sequence
    return news, olds


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _quotient(a, b):
    # a correctly rounded division by a constant (a scalar divisor may become a product with its reciprocal)
    return a / torch.full_like(a, b)


def _nibbles(x):
    """Nibbles c + 8 (uint8) of symmetric 4-bit codes of x [..., D], and the scale of every head."""
    s = _quotient(x.abs().amax(-1), 7.0)
    q = torch.where(s.unsqueeze(-1) > 0, (x / s.unsqueeze(-1)).round_().clamp_(-8, 7), torch.zeros_like(x))
    return (q + 8.0).to(torch.uint8), s


def _pages(g, pages, heads, page, dim, dtype, keys):
    """A cache's pages of keys or values, filled."""
    codes = torch.empty((pages, heads, page, dim // 2) if keys else (pages, heads, page // 16, 8 * dim),
                        dtype=torch.uint8, device="cuda")
    scales = torch.empty((pages, heads, page), device="cuda")
    # keys have channels that stand out, the same for every token of a head
    lift = torch.randn((heads, 1, dim), generator=g, device="cuda") if keys else 0.0
    step = max(1, (1 << 25) // (heads * page * dim))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        x = (torch.randn((n, heads, page, dim), generator=g, device="cuda") + lift).to(dtype).float()
        u, scales[at:at + n] = _nibbles(x)
        if keys:
            codes[at:at + n] = u[..., 0::2] | (u[..., 1::2] << 4)
        else:
            u = u.view(n, heads, page // 16, 4, 4, dim // 32, 2, 16).permute(0, 1, 2, 3, 7, 5, 4, 6)
            codes[at:at + n] = (u[..., 0] | (u[..., 1] << 4)).reshape(n, heads, page // 16, 8 * dim)
    return codes, scales


def _cache(g, pages, heads, page, dim, dtype):
    return (*_pages(g, pages, heads, page, dim, dtype, True), *_pages(g, pages, heads, page, dim, dtype, False))


def prepare(case, seed):
    g = _gen(seed)
    state = dict(case)
    dtype, dim, op = getattr(torch, case["dtype"]), case["dim"], case["op"]
    if op in ("rope", "append"):
        half = case["rotary"] // 2
        at = torch.arange(half, dtype=torch.float64, device="cuda")
        state["freq"] = 10000.0 ** (-at / half) / case["stretch"]
    if op == "rope":
        t = case["tokens"]
        state["x"] = torch.randn((t, case["heads"], dim), generator=g, device="cuda").to(dtype)
        state["positions"] = case["first"] + torch.arange(t, device="cuda")
        return state
    if op == "attend":
        news, olds = _lengths(case)
        longest, page = max(olds), case["page"]
        cols = max(1, -(-longest // page))
        need = [-(-n // page) for n in olds]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device="cuda").int()
        table = torch.zeros((len(olds), cols), dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        state["cache"] = _cache(g, pages, case["kv_heads"], page, dim, dtype)
        state["table"] = table
        state["news"], state["olds"] = news, olds
        state["kv_lens"] = torch.tensor(olds, dtype=torch.int32, device="cuda")
        ends = [0]
        for n in news:
            ends.append(ends[-1] + n)
        state["cu_q"] = None if max(news) == 1 else torch.tensor(ends, dtype=torch.int32, device="cuda")
        state["x"] = (1.3 * torch.randn((ends[-1], case["heads"], dim), generator=g, device="cuda")).to(dtype)
        return state
    t, page, kv = case["tokens"], case["page"], case["kv_heads"]
    if op == "append":
        # queries, keys and values as one projection writes them
        rows = torch.randn((t, case["heads"] + 2 * kv, dim), generator=g, device="cuda")
        rows[:, case["heads"]:case["heads"] + kv] += torch.randn((kv, dim), generator=g, device="cuda")
        state["rows"] = rows.to(dtype)
        state["positions"] = case["first"] + (torch.arange(t, device="cuda") if case["prompt"] else
                                              torch.randint(0, 4096, (t,), generator=g, device="cuda"))
    spread = op == "append" and not case["prompt"]         # one token of each sequence, on a page of its own
    pages = (t if spread else -(-t // page)) + 2
    order = torch.randperm(pages, generator=g, device="cuda")
    at = torch.arange(t, device="cuda")
    if spread:
        slots = order[:t] * page + torch.randint(0, page, (t,), generator=g, device="cuda")
    else:
        slots = order[at // page] * page + at % page
    if case.get("padded"):
        slots[t - case["padded"]:] = -1                   # padding is not stored
    state["slots"] = slots
    state["cache"] = _cache(g, pages, kv, page, dim, dtype)
    return state


# ---------------------------------------------------------------- plain forms

def _plain_rope(x, positions, freq, interleaved):
    # angles of far positions, and values next to a border of 4-bit codes: 64 bits
    turn = positions.double().unsqueeze(-1) * freq
    cos, sin = torch.cos(turn).unsqueeze(1), torch.sin(turn).unsqueeze(1)
    n = 2 * freq.numel()
    v = x.double()
    a, b = (v[..., 0:n:2], v[..., 1:n:2]) if interleaved else (v[..., :n // 2], v[..., n // 2:n])
    pair = (a * cos - b * sin, b * cos + a * sin)
    done = torch.stack(pair, -1).flatten(-2) if interleaved else torch.cat(pair, -1)
    return torch.cat((done, v[..., n:]), -1)


def _plain_keys(codes, scales):
    """[..., page, D/2], [..., page] -> values [..., page, D]"""
    u = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    return (u.float() - 8.0) * scales.unsqueeze(-1)


def _plain_values(codes, scales):
    """[..., page/16, 8 D], [..., page] -> values [..., page, D]"""
    dim = codes.shape[-1] // 8
    u = torch.stack((codes & 15, codes >> 4), -1)
    u = u.view(*codes.shape[:-1], 4, 16, dim // 32, 4, 2)              # g, r, v, i, half
    n = u.dim()
    u = u.permute(*range(n - 5), n - 5, n - 2, n - 3, n - 1, n - 4)    # g, i, v, half, r
    u = u.reshape(*codes.shape[:-2], codes.shape[-2] * 16, dim)
    return (u.float() - 8.0) * scales.unsqueeze(-1)


def _plain_append(s):
    hq, kv = s["heads"], s["kv_heads"]
    q, k, v = s["rows"][:, :hq], s["rows"][:, hq:hq + kv], s["rows"][:, hq + kv:]
    turned = _plain_rope(q, s["positions"], s["freq"], s["interleaved"]).to(q.dtype)
    ku, ks = _nibbles(_plain_rope(k, s["positions"], s["freq"], s["interleaved"]).float())
    vu, vs = _nibbles(v.float())
    n = s["tokens"] - s["padded"]                          # (padding is at the end, and is not stored)
    dim, page = k.shape[2], s["page"]
    at, off = s["slots"][:n] // page, s["slots"][:n] % page
    k_codes, k_scales, v_codes, v_scales = s["cache"]
    k_codes[at, :, off] = (ku[..., 0::2] | (ku[..., 1::2] << 4))[:n]
    k_scales[at, :, off] = ks[:n]
    v_scales[at, :, off] = vs[:n]
    lanes = v_codes.view(v_codes.shape[0], kv, page // 16, 4, 16, dim // 32, 4)
    by = vu[:n].view(n, kv, dim // 32, 2, 16)
    by = (by[:, :, :, 0] | (by[:, :, :, 1] << 4)).transpose(2, 3)      # [n, heads, r, v]
    lanes[at, :, off // 16, off % 16 // 4, :, :, off % 4] = by
    k_out, v_out = _plain_read(s["cache"], s["slots"], q.dtype)
    return turned, k_out, v_out


def _plain_read(cache, slots, dtype):
    k_codes, k_scales, v_codes, v_scales = cache
    page = k_codes.shape[2]
    live = (slots >= 0).view(-1, 1, 1)
    at, off = slots.clamp_min(0) // page, slots.clamp_min(0) % page
    dim = 2 * k_codes.shape[3]
    k = _plain_keys(k_codes[at, :, off], k_scales[at, :, off])
    lanes = v_codes.view(v_codes.shape[0], v_codes.shape[1], page // 16, 4, 16, dim // 32, 4)
    by = lanes[at, :, off // 16, off % 16 // 4, :, :, off % 4]          # [t, heads, r, v]
    u = torch.stack((by & 15, by >> 4), -1).permute(0, 1, 3, 4, 2).flatten(-3)
    v = (u.float() - 8.0) * v_scales[at, :, off].unsqueeze(-1)
    zero = torch.zeros((), device=k.device)
    return torch.where(live, k, zero).to(dtype), torch.where(live, v, zero).to(dtype)


def _plain_softmax(scores, seen):
    scores = torch.where(seen, scores, torch.full((), -math.inf, device=scores.device))
    p = torch.exp(scores - scores.amax(-1, keepdim=True).nan_to_num(neginf=0.0))
    return p / p.sum(-1, keepdim=True).clamp_min(1e-30)


def _plain_attend(s):
    q, cache, table, news, olds = s["x"], s["cache"], s["table"], s["news"], s["olds"]
    heads, kv, dim, page = s["heads"], s["kv_heads"], s["dim"], s["page"]
    share, scale = heads // kv, 1.0 / math.sqrt(dim)
    back = s["window"] if s["window"] else 1 << 30
    if s["cu_q"] is None:                                  # one query a sequence: all of them at once
        b, cols = table.shape
        at = table.flatten().long()
        k = _plain_keys(cache[0][at], cache[1][at]).view(b, cols, kv, page, dim).transpose(1, 2).flatten(2, 3)
        v = _plain_values(cache[2][at], cache[3][at]).view(b, cols, kv, page, dim).transpose(1, 2).flatten(2, 3)
        x = q.float().view(b, kv, share, dim) * scale
        key = torch.arange(cols * page, device=q.device)
        n = s["kv_lens"].view(b, 1, 1, 1)
        p = _plain_softmax(torch.matmul(x, k.transpose(-1, -2)), (key < n) & (key >= n - back))
        return torch.matmul(p, v).view(b, heads, dim).to(q.dtype)
    out, start = torch.empty_like(q), 0
    for b, (new, old) in enumerate(zip(news, olds)):
        at = table[b, :max(1, -(-old // page))].long()
        k = _plain_keys(cache[0][at], cache[1][at]).transpose(0, 1).flatten(1, 2)
        v = _plain_values(cache[2][at], cache[3][at]).transpose(0, 1).flatten(1, 2)
        key = torch.arange(k.shape[1], device=q.device)
        here = (old - new + torch.arange(new, device=q.device)).unsqueeze(-1)
        seen = (key <= here) & (key > here - back)
        x = q[start:start + new].float() * scale
        for h in range(kv):                                # (scores of one key head at a time, for the memory)
            mine = slice(h * share, (h + 1) * share)
            p = _plain_softmax(torch.matmul(x[:, mine].transpose(0, 1), k[h].t()), seen)
            out[start:start + new, mine] = torch.matmul(p, v[h]).transpose(0, 1).to(q.dtype)
        start += new
    return out


def run(state):
    op = state["op"]
    if not own:
        if op == "rope":
            return _plain_rope(state["x"], state["positions"], state["freq"], state["interleaved"]).to(state["x"].dtype)
        if op == "append":
            return _plain_append(state)
        if op == "read":
            return _plain_read(state["cache"], state["slots"], getattr(torch, state["dtype"]))
        return _plain_attend(state)
    from w4a4_group_quantized_amd import apex4
    if op == "rope":
        return apex4.rope(state["x"], state["positions"], state["freq"], interleaved=state["interleaved"])
    if op == "append":
        hq, kv, rows = state["heads"], state["kv_heads"], state["rows"]
        q = apex4.kv4_append(state["cache"], rows[:, hq:hq + kv], rows[:, hq + kv:], state["slots"], q=rows[:, :hq],
                             positions=state["positions"], inv_freq=state["freq"], interleaved=state["interleaved"])
        return (q, *apex4.kv4_read(state["cache"], state["slots"], rows.dtype))     # the values that the codes are
    if op == "read":
        return apex4.kv4_read(state["cache"], state["slots"], getattr(torch, state["dtype"]))
    return apex4.kv4_attention(state["x"], state["cache"], state["table"], state["kv_lens"], state["cu_q"],
                               window=state["window"], max_q=max(state["news"]), max_kv=max(state["olds"]))


# ---------------------------------------------------------------- work

def work(case):
    op, dim = case["op"], case["dim"]
    size = 4 if case["dtype"] == "float32" else 2
    if op == "rope":
        t, h = case["tokens"], case["heads"]
        return {"bytes": 2 * size * t * h * dim + 8 * t + 4 * case["rotary"], "flops": 3.0 * t * h * case["rotary"]}
    if op == "read":
        t, h = case["tokens"], case["kv_heads"]
        return {"bytes": t * h * (dim + 8) + 2 * size * t * h * dim + 8 * t, "flops": 4.0 * t * h * dim}
    if op == "append":
        t, h, kv = case["tokens"], case["heads"], case["kv_heads"]
        live = t - case["padded"]
        once = 2 * size * t * h * dim + 2 * size * live * kv * dim + live * kv * (dim + 8)     # rotate and store
        back = live * kv * (dim + 8) + 2 * size * t * kv * dim                                 # and read back
        return {"bytes": once + back + 24 * t, "flops": 3.0 * t * (h + kv) * case["rotary"] + 8.0 * live * kv * dim}
    news, olds = _lengths(case)
    back = case["window"] if case["window"] else 1 << 30
    pairs = keys = 0
    for new, old in zip(news, olds):
        ends = range(old - new + 1, old + 1)
        pairs += sum(max(0, min(e, back)) for e in ends)
        keys += min(old, back + new - 1)
    each = 2 * size * sum(news) * case["heads"] * dim
    return {"bytes": keys * case["kv_heads"] * (dim + 8) + each, "flops": 4.0 * pairs * case["heads"] * dim}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_rope(x, positions, freq, interleaved):
    half = freq.numel()
    wave = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                       positions.to(torch.float64)[:, None, None] * freq)
    y = x.to(torch.float64).clone()
    if interleaved:
        z = torch.view_as_complex(y[..., :2 * half].reshape(*x.shape[:-1], half, 2).contiguous()) * wave
        y[..., :2 * half] = torch.view_as_real(z).reshape(*x.shape[:-1], 2 * half)
    else:
        z = torch.complex(y[..., :half].contiguous(), y[..., half:2 * half].contiguous()) * wave
        y[..., :half], y[..., half:2 * half] = z.real, z.imag
    return y


def _exact_codes(x):
    """The values that 4-bit codes of x stand for (x: 32-bit numbers held in 64)."""
    s = (x.abs().max(-1, keepdim=True).values / 7).float().double()
    c = torch.nan_to_num((x / s).float().double().round(), nan=0.0).clamp(-8, 7)
    return c * s


def _exact_tokens(cache, slots):
    """Keys and values of the slots, nibble by nibble from their places."""
    k_codes, k_scales, v_codes, v_scales = cache
    page, dim = k_codes.shape[2], 2 * k_codes.shape[3]
    at, off = (slots // page).view(-1, 1, 1), (slots % page).view(-1, 1, 1)
    head = torch.arange(k_codes.shape[1], device=slots.device).view(1, -1, 1)
    d = torch.arange(dim, device=slots.device).view(1, 1, -1)
    k = (k_codes[at, head, off, d // 2].to(torch.int64) // torch.where(d % 2 == 1, 16, 1)) % 16
    place = (off % 16 // 4 * 16 + d % 16) * (dim // 8) + d // 32 * 4 + off % 4
    v = (v_codes[at, head, off // 16, place].to(torch.int64) // torch.where(d % 32 >= 16, 16, 1)) % 16
    ks, vs = k_scales[at, head, off].double(), v_scales[at, head, off].double()
    return (k - 8).double() * ks, (v - 8).double() * vs


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _exact_rope(s["x"], s["positions"], s["freq"], s["interleaved"])
    if op == "append":
        hq, kv, rows = s["heads"], s["kv_heads"], s["rows"]
        turned = _exact_rope(rows[:, :hq + kv], s["positions"], s["freq"], s["interleaved"])
        live = (s["slots"] >= 0).view(-1, 1, 1).double()
        return (turned[:, :hq], _exact_codes(turned[:, hq:].float().double()) * live,
                _exact_codes(rows[:, hq + kv:].double()) * live)
    if op == "read":
        parts = [_exact_tokens(s["cache"], slots) for slots in s["slots"].split(4096)]
        return tuple(torch.cat(p) for p in zip(*parts))
    q, table, page = s["x"].double(), s["table"].long(), s["page"]
    share = s["heads"] // s["kv_heads"]
    out, start = torch.zeros(q.shape, dtype=torch.float64, device=q.device), 0
    for b, (new, old) in enumerate(zip(s["news"], s["olds"])):
        if old:
            key = torch.arange(old, device=q.device)
            k, v = _exact_tokens(s["cache"], table[b, key // page] * page + key % page)
            for h in range(s["heads"]):
                scores = q[start:start + new, h] @ k[:, h // share].T / math.sqrt(s["dim"])
                ahead = key - torch.arange(old - new, old, device=q.device).unsqueeze(1)
                gone = (ahead > 0) | (ahead <= -s["window"]) if s["window"] else ahead > 0
                out[start:start + new, h] = torch.softmax(scores.masked_fill(gone, -math.inf), -1) @ v[:, h // share]
        start += new
    return out
