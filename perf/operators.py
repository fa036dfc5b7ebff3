"""Operators of sparse and 8-bit layers, as cases to measure.

Three operators: routing tokens to experts ("route"), the experts' W4A4
feed-forward network over routed tokens ("experts"), and the linear layer in
8-bit floating point with a scale for each block of 128 ("e4m3").  With
`own` false, `run` computes them from elementary torch operations; with
`own` true it calls this repository's entry points.
"""
import math

import torch

own = False

GROUP = 128


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token of a decoding step, a small layer: latency
        dict(name="route-token", op="route", tokens=1, experts=64, k=6, score="softmax", bias=False, groups=1,
             keep=1, top=1, renormalize=True, scale=1.0, dtype="float32", padded=0),
        # a ragged batch of short prompts with padding; the number of experts is no power of two
        dict(name="route-batch", op="route", tokens=777, experts=160, k=6, score="softmax", bias=False, groups=8,
             keep=3, top=1, renormalize=False, scale=16.0, dtype="bfloat16", padded=33),
        # a long prefill with a balancing bias and groups of experts
        dict(name="route-prefill", op="route", tokens=16384, experts=256, k=8, score="sigmoid", bias=True, groups=8,
             keep=4, top=2, renormalize=True, scale=2.5, dtype="float32", padded=0),
        # one token through experts of an eighth of the 4096/11008 layer's width: every chosen expert has one row
        dict(name="experts-token", op="experts", tokens=1, experts=64, k=8, hidden=4096, inter=1408, padded=0),
        # a decoding batch with padded places: most experts have a row or two
        dict(name="experts-decode", op="experts", tokens=27, experts=64, k=6, hidden=4096, inter=1408, padded=3),
        # a short prompt through eight wide experts
        dict(name="experts-wide", op="experts", tokens=301, experts=8, k=2, hidden=4096, inter=11008, padded=0),
        # a long prefill through many narrow experts
        dict(name="experts-prefill", op="experts", tokens=4096, experts=64, k=8, hidden=4096, inter=1408, padded=0),
        # the 4096-wide output projection for one token
        dict(name="e4m3-token", op="e4m3", tokens=1, n=4096, k=4096, dtype="bfloat16"),
        # the 28672 -> 8192 down projection for a decoding batch
        dict(name="e4m3-decode", op="e4m3", tokens=16, n=8192, k=28672, dtype="float16"),
        # the 8192 -> 28672 up projection for a large decoding batch
        dict(name="e4m3-batch", op="e4m3", tokens=64, n=28672, k=8192, dtype="bfloat16"),
        # a ragged prompt, rows and columns that end inside a tile and a block
        dict(name="e4m3-ragged", op="e4m3", tokens=515, n=4008, k=11008, dtype="float16"),
        # the 8192 -> 10240 fused projection of a long prefill
        dict(name="e4m3-prefill", op="e4m3", tokens=4096, n=10240, k=8192, dtype="bfloat16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("route", "experts", "experts", "e4m3", "e4m3"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        experts = groups * _log_int(rng, max(2, 8 // groups), 512 // groups)
        keep = rng.randint((groups + 1) // 2, groups)
        most = keep * (experts // groups)
        tokens = _log_int(rng, 1, max(1, min(16384, 16384 * 256 // experts)))
        bias = rng.random() < 0.5
        return dict(op=op, tokens=tokens, experts=experts, k=min(most, _log_int(rng, 1, 8)),
                    score=rng.choice(("softmax", "sigmoid")), bias=bias, groups=groups, keep=keep,
                    top=rng.choice((1, 2)), renormalize=rng.random() < 0.5, scale=rng.choice((1.0, 2.5)),
                    dtype=rng.choice(("float32", "float16", "bfloat16")),
                    padded=rng.randint(0, tokens // 4))
    if op == "experts":
        experts = _log_int(rng, 4, 128)
        k = min(experts, rng.randint(1, 8))
        hidden = 128 * _log_int(rng, 4, 64)
        # at most the weights of the widest listed case, at most the products of the longest
        inter = 128 * _log_int(rng, 2, max(2, min(86, 8 * 4096 * 11008 // (experts * hidden * 128))))
        most = 4096 * 8 * 4096 * 1408 // (k * hidden * inter)
        tokens = _log_int(rng, 1, max(1, min(4096, most)))
        return dict(op=op, tokens=tokens, experts=experts, k=k, hidden=hidden, inter=inter,
                    padded=rng.randint(0, tokens // 4))
    k = 128 * _log_int(rng, 2, 224)
    n = _log_int(rng, 64, min(28672, 8192 * 28672 // k))
    tokens = _log_int(rng, 1, max(1, min(4096, 4096 * 10240 * 8192 // (n * k))))
    return dict(op=op, tokens=tokens, n=n, k=k, dtype=rng.choice(("float16", "bfloat16")))


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(g, rows, cols, dtype):
    """N(0, 1) with one channel in a hundred, the same for every token, twenty times as large."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    big = torch.rand((cols,), generator=g, device="cuda") < 0.01
    return torch.where(big, 20.0 * x, x).to(dtype)


def _router_logits(g, tokens, experts):
    """Scores of a router: some experts are liked by all tokens."""
    liked = 0.5 * torch.randn((experts,), generator=g, device="cuda")
    return 1.5 * torch.randn((tokens, experts), generator=g, device="cuda") + liked


def _quotient(a, b):
    # a correctly rounded division by a constant (a scalar divisor may become a product with its reciprocal)
    return a / torch.full_like(a, b)


def _pack_int4(w):
    """Symmetric 4-bit codes, two a byte (even index in the low nibble), and the scale of every 128."""
    v = w.unflatten(-1, (-1, GROUP))
    s = _quotient(v.abs().amax(-1), 7.0)
    q = (v / s.unsqueeze(-1)).round_().clamp_(-8, 7).nan_to_num_(0.0).to(torch.int8).flatten(-2)
    return ((q[..., 0::2] & 15) | ((q[..., 1::2] & 15) << 4)).view(torch.uint8).contiguous(), s


def prepare(case, seed):
    g = _gen(seed)
    state = dict(case)
    if case["op"] == "route":
        t, e = case["tokens"], case["experts"]
        logits = _router_logits(g, t, e)
        if case["padded"]:
            logits[t - case["padded"]:] = -math.inf       # padding routes nowhere
        state["logits"] = logits.to(getattr(torch, case["dtype"]))
        state["balance"] = 0.1 * torch.randn((e,), generator=g, device="cuda") if case["bias"] else None
    elif case["op"] == "experts":
        t, e, k, hid, mid = (case[n] for n in ("tokens", "experts", "k", "hidden", "inter"))
        state["x"] = _activations(g, t, hid, torch.float16)
        gates, ids = torch.softmax(_router_logits(g, t, e), -1).topk(k, -1)
        ids = ids.to(torch.int32)
        if case["padded"]:
            ids[t - case["padded"]:] = -1
        state["ids"], state["gates"] = ids, (gates / gates.sum(-1, keepdim=True)).contiguous()
        for name, n, kk in (("gate_up", 2 * mid, hid), ("down", hid, mid)):
            q = torch.empty((e, n, kk // 2), dtype=torch.uint8, device="cuda")
            s = torch.empty((e, n, kk // GROUP), device="cuda")
            for i in range(e):
                w = torch.randn((n, kk), generator=g, device="cuda").mul_(0.02).half().float()
                q[i], s[i] = _pack_int4(w)
            state[name], state[name + "_scales"] = q, s
        # the most rows that one expert gets: the room of the plain form's batch
        state["room"] = int(torch.bincount(ids[ids >= 0].long(), minlength=1).max()) if t > case["padded"] else 1
    else:
        dtype = getattr(torch, case["dtype"])
        state["x"] = _activations(g, case["tokens"], case["k"], dtype)
        w = torch.randn((case["n"], case["k"]), generator=g, device="cuda").mul_(0.02).to(dtype).float()
        n, kb = case["n"], case["k"] // GROUP
        rows = -(-n // GROUP)
        tiles = torch.nn.functional.pad(w, (0, 0, 0, rows * GROUP - n)).view(rows, GROUP, kb, GROUP)
        s = _quotient(tiles.abs().amax((1, 3)), 448.0)
        q = (tiles / s[:, None, :, None]).clamp_(-448.0, 448.0).reshape(rows * GROUP, -1)[:n]
        state["w"] = q.to(torch.float8_e4m3fn).view(torch.uint8).contiguous()
        state["w_scales"] = s
    return state


# ---------------------------------------------------------------- plain forms

def _plain_route(logits, k, score, bias, groups, keep, top, renormalize, scale):
    t, e = logits.shape
    x = logits.double()                                   # ranks go by values next to each other
    x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
    if score == "softmax":
        high = x.amax(-1, keepdim=True).nan_to_num(neginf=0.0)
        p = torch.exp(x - high)
        p = p / p.sum(-1, keepdim=True).clamp_min(1e-300)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    key = x if bias is None else torch.where(torch.isneginf(x), x, p + bias.double())
    if groups > 1:
        by = key.view(t, groups, e // groups)
        if top == 1:
            of = by.amax(-1)
        else:
            each = by if bias is not None else torch.where(torch.isneginf(by), by, p.view_as(by))
            two = each.sort(-1, descending=True).values[..., :2]
            live = ~torch.isneginf(two)
            of = torch.where(live, two, torch.zeros_like(two)).sum(-1)
            of = torch.where(live.any(-1), of, torch.full_like(of, -math.inf))
        best = of.sort(dim=-1, descending=True, stable=True).indices[:, :keep]
        kept = torch.zeros((t, groups), dtype=torch.bool, device=x.device).scatter_(1, best, True)
        key = torch.where(kept.unsqueeze(-1), by, torch.full_like(by, -math.inf)).view(t, e)
    order = key.sort(dim=-1, descending=True, stable=True)
    ids, live = order.indices[:, :k], ~torch.isneginf(order.values[:, :k])
    chosen = torch.where(live, p.gather(1, ids), torch.zeros((), dtype=p.dtype, device=p.device))
    if renormalize:
        chosen = chosen / chosen.sum(-1, keepdim=True).clamp_min(1e-300)
    return torch.where(live, ids, torch.full_like(ids, -1)).int(), (chosen * scale).float()


def _int4_values(x):
    """The values that symmetric 4-bit codes with a scale for every 128 stand for."""
    v = x.float().unflatten(-1, (-1, GROUP))
    a = v.abs().amax(-1, keepdim=True)
    s = _quotient(a, 7.0)
    q = torch.where(a > 0, torch.clamp(torch.round(v / s), -8, 7), torch.zeros_like(v))
    return (q * s).flatten(-2)


def _unpack(q, s):
    low, high = (q << 4).view(torch.int8) >> 4, q.view(torch.int8) >> 4
    codes = torch.stack((low, high), -1).flatten(-2).float()
    return (codes.unflatten(-1, (-1, GROUP)) * s.unsqueeze(-1)).flatten(-2)


def _plain_experts(x, ids, gates, gate_up, gate_up_scales, down, down_scales, room):
    t, k = ids.shape
    e, mid = gate_up.shape[0], gate_up.shape[1] // 2
    flat = ids.reshape(-1).long()
    live = (flat >= 0) & (flat < e)
    # the place of every slot: its expert, and its rank among the expert's slots; slots without an expert share
    # the last place of expert 0
    hot = (flat.unsqueeze(1) == torch.arange(e, device=x.device)).int()
    expert = torch.where(live, flat, torch.zeros_like(flat))
    rank = (hot.cumsum(0) - hot).gather(1, expert.unsqueeze(1)).squeeze(1)
    place = expert * (room + 1) + torch.where(live, rank, torch.full_like(rank, room))
    token = torch.arange(t * k, device=x.device) // k
    rows = torch.zeros((e * (room + 1), x.shape[1]), device=x.device)
    rows[place] = _int4_values(x)[token]
    rows = rows.view(e, room + 1, -1).transpose(1, 2).contiguous()
    both = torch.bmm(_unpack(gate_up, gate_up_scales), rows)              # [E, 2I, room + 1]
    gate, up = both[:, :mid], both[:, mid:]
    h = (gate / (1.0 + torch.exp(-gate)) * up).clamp(-65504.0, 65504.0).transpose(1, 2).contiguous().half()
    out = torch.bmm(_unpack(down, down_scales), _int4_values(h).transpose(1, 2).contiguous())
    out = out.transpose(1, 2).reshape(e * (room + 1), -1)[place]
    weight = torch.where(live, gates.reshape(-1), torch.zeros((), device=x.device)).unsqueeze(1)
    return (weight * out).view(t, k, -1).sum(1).half()


def _plain_e4m3(x, w, w_scales):
    v = x.float().unflatten(-1, (-1, GROUP))
    s = _quotient(v.abs().amax(-1, keepdim=True), 448.0)
    q = torch.where(s > 0, torch.clamp(v / s, -448.0, 448.0), torch.zeros_like(v)).to(torch.float8_e4m3fn).float()
    a = (q * s).flatten(-2)
    scales = w_scales.repeat_interleave(GROUP, 0)[: w.shape[0]].repeat_interleave(GROUP, 1)
    b = w.view(torch.float8_e4m3fn).float() * scales
    return torch.mm(a, b.t().contiguous()).to(x.dtype)


def run(state):
    if state["op"] == "route":
        if own:
            from w4a4_group_quantized_amd import apex4
            return apex4.route(state["logits"], state["k"], score=state["score"], bias=state["balance"],
                               n_group=state["groups"], topk_group=state["keep"], group_top=state["top"],
                               renormalize=state["renormalize"], scale=state["scale"])
        return _plain_route(state["logits"], state["k"], state["score"], state["balance"], state["groups"],
                            state["keep"], state["top"], state["renormalize"], state["scale"])
    if state["op"] == "experts":
        args = (state["x"], state["ids"], state["gates"], state["gate_up"], state["gate_up_scales"], state["down"],
                state["down_scales"])
        if own:
            from w4a4_group_quantized_amd import apex4
            return apex4.experts(*args)
        return _plain_experts(*args, state["room"])
    if own:
        from w4a4_group_quantized_amd import apex4
        return apex4.linear_e4m3(state["x"], state["w"], state["w_scales"])
    return _plain_e4m3(state["x"], state["w"], state["w_scales"])


# ---------------------------------------------------------------- work

def work(case):
    if case["op"] == "route":
        t, e = case["tokens"], case["experts"]
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": t * e * size + (4 * e if case["bias"] else 0) + 8 * t * case["k"], "flops": 4.0 * t * e}
    if case["op"] == "experts":
        t, e, k, hid, mid = (case[n] for n in ("tokens", "experts", "k", "hidden", "inter"))
        live = t - case["padded"]
        used = e * (1.0 - (1.0 - k / e) ** live)          # experts with a row, of evenly spread choices
        weights = used * 3 * hid * mid * (0.5 + 4.0 / GROUP)
        return {"bytes": weights + 4 * t * hid + 8 * t * k, "flops": 6.0 * live * k * hid * mid}
    t, n, k = case["tokens"], case["n"], case["k"]
    scales = 4 * (k // GROUP) * -(-n // GROUP)
    return {"bytes": n * k + scales + 2 * t * k + 2 * t * n, "flops": 2.0 * t * n * k}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_route(s):
    x = s["logits"].to(torch.float64).cpu()
    bias = None if s["balance"] is None else s["balance"].to(torch.float64).cpu()
    t, e = x.shape
    dead = torch.isnan(x) | (x == -math.inf)
    if s["score"] == "softmax":
        p = torch.softmax(x.masked_fill(dead, -math.inf), -1).masked_fill(dead, 0.0)
    else:
        p = torch.special.expit(x).masked_fill(dead, 0.0)
    key = (x if bias is None else p + bias).masked_fill(dead, -math.inf)
    if s["groups"] > 1:
        size = e // s["groups"]
        value = key if bias is not None or s["top"] == 1 else p.masked_fill(dead, -math.inf)
        score = []
        for i in range(s["groups"]):
            best = value[:, i * size:(i + 1) * size].topk(min(s["top"], size), -1).values
            total = best.masked_fill(best == -math.inf, 0.0).sum(-1)
            score.append(total.masked_fill((best == -math.inf).all(-1), -math.inf))
        score = torch.stack(score, -1)
        # a group's place is the number of groups before it: better ones, and equal ones of lower index
        for i in range(s["groups"]):
            ahead = (score > score[:, i:i + 1]).sum(-1) + (score[:, :i] == score[:, i:i + 1]).sum(-1)
            key[:, i * size:(i + 1) * size].masked_fill_((ahead >= s["keep"]).unsqueeze(-1), -math.inf)
    ids = torch.full((t, s["k"]), -1, dtype=torch.int32)
    gates = torch.zeros((t, s["k"]), dtype=torch.float64)
    rows = torch.arange(t)
    for j in range(s["k"]):
        best = key.amax(-1)
        at = (key == best.unsqueeze(-1)).to(torch.uint8).argmax(-1)       # the first of the best
        live = best > -math.inf
        ids[live, j] = at[live].int()
        gates[live, j] = p[rows, at][live]
        key[rows, at] = -math.inf
    if s["renormalize"]:
        total = gates.sum(-1, keepdim=True)
        gates = torch.where(total > 0, gates / total, torch.zeros_like(gates))
    return ids, gates * s["scale"]


def _exact_codes(x, most):
    """(quotients by the scale of each 128, as 32-bit numbers; the scales), from the definition."""
    rows, cols = x.shape
    v = x.double().reshape(rows, cols // GROUP, GROUP)
    scale = (v.abs().max(-1, keepdim=True).values / most).float().double()
    return torch.nan_to_num((v / scale).float().double(), nan=0.0, posinf=0.0, neginf=0.0), scale


def _exact_int4(x):
    q, s = _exact_codes(x, torch.tensor(7.0, dtype=torch.float64, device=x.device))
    return (q.round().clamp(-8, 7) * s).reshape(x.shape)


def _exact_weight(q, s):
    w = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.float64, device=q.device)
    n = q.to(torch.int64)
    for half, v in ((0, n % 16), (1, n // 16)):
        w[:, half::2] = (v - 16 * (v > 7)).double()
    for j in range(s.shape[1]):
        w[:, GROUP * j:GROUP * (j + 1)] *= s[:, j:j + 1].double()
    return w


def _exact_experts(s):
    x, ids, gates = s["x"], s["ids"], s["gates"].double()
    mid = s["gate_up"].shape[1] // 2
    xv = _exact_int4(x)
    y = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    for e in range(s["gate_up"].shape[0]):
        token, slot = (ids == e).nonzero(as_tuple=True)
        if not token.numel():
            continue
        both = xv[token] @ _exact_weight(s["gate_up"][e], s["gate_up_scales"][e]).T
        a, b = both[:, :mid], both[:, mid:]
        h = (a * torch.sigmoid(a) * b).clamp(-65504, 65504).half()
        d = _exact_int4(h) @ _exact_weight(s["down"][e], s["down_scales"][e]).T
        y.index_add_(0, token, gates[token, slot].unsqueeze(1) * d)
    return y


def _exact_e4m3(s):
    x, w = s["x"], s["w"].to(torch.int64)
    q, sa = _exact_codes(x, torch.tensor(448.0, dtype=torch.float64, device=x.device))
    # nearest 8-bit number, ties to even: three bits after the leading one, no exponent below -6
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))).clamp_min(-6.0) - 3.0)
    a = (torch.round(q / step) * step).clamp(-448, 448) * sa
    power, part = (w >> 3) & 15, (w & 7).double()
    value = torch.where(power == 0, part * 2.0 ** -9, (8 + part) * torch.exp2(power.double() - 10.0))
    value = torch.where(w >= 128, -value, value)
    out = torch.zeros((x.shape[0], w.shape[0]), dtype=torch.float64, device=x.device)
    at = torch.arange(w.shape[0], device=x.device) // GROUP
    for j in range(sa.shape[1]):
        out += (a[:, j] @ value[:, GROUP * j:GROUP * (j + 1)].T) * s["w_scales"][at, j].double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s)
    return _exact_experts(s) if case["op"] == "experts" else _exact_e4m3(s)
