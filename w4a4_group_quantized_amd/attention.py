"""The attention half of a W4A4 decoder layer: rotary positions, a paged key/value
cache in 4 bits, and attention over it.

`rope_frequencies` makes the frequencies that apex4.rope and apex4.kv4_append take,
scaled for longer contexts where that is asked for.  `KVCache4` holds the pages of
one layer.  `BatchPlan` says where a step's tokens stand and are kept; a batch has
one for all its layers.  `CachedLayerW4A4` is `LlamaLayerW4A4` with attention in
place of its stand-in.

None of them keeps a workspace: a call takes its own from torch's caching
allocator, so calls on different streams do not share one.
"""
from __future__ import annotations

import math

import torch

from . import apex4
from .linear import LlamaLayerW4A4


def rope_frequencies(rotary: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                     original: int = 4096, low: float = 1.0, high: float | None = None, device="cuda"):
    """(frequencies float64 [rotary / 2], the factor that goes with them) of rotary positions,
    base^(-2 i / rotary) with

    scaling None: as they are; "linear": divided by `factor`; "ntk": a base grown so that the
    slowest turns `factor` times slower and the fastest stays; "wavelength": divided by `factor`
    where a turn takes more than original / low positions, as they are where it takes less than
    original / high, and blended between (high 4 when None); "yarn": divided by `factor` where there
    are fewer than `low` turns in `original` positions, as they are from `high` on (32 when None),
    blended by the pair's number between, with a factor 0.1 ln(factor) + 1 for queries and
    keys (1 otherwise): the `scale` of apex4.rope, the `rope_scale` of apex4.kv4_append.
    """
    if rotary < 16 or rotary % 16 or not factor >= 1.0:
        raise ValueError(f"rotary must be a multiple of 16 and factor at least 1, got {rotary, factor}")
    if high is None:
        high = 32.0 if scaling == "yarn" else 4.0
    if not base > (1.0 if scaling == "yarn" else 0.0):
        raise ValueError(f"base must be above 0 (yarn: above 1), got {base}")
    if scaling in ("wavelength", "yarn") and not (0.0 < low < high and original > 0):
        raise ValueError(f"0 < low < high and original > 0 are needed, got {low, high, original}")
    half = rotary // 2
    pair = torch.arange(half, dtype=torch.float64)
    scale = 1.0
    if scaling == "ntk":
        base = base * factor ** (rotary / (rotary - 2))
    freqs = base ** (-pair / half)
    if scaling == "linear":
        freqs = freqs / factor
    elif scaling == "wavelength":
        turns = original * freqs / (2 * math.pi)             # in `original` positions
        keep = ((turns - low) / (high - low)).clamp(0.0, 1.0)
        freqs = freqs * (keep + (1 - keep) / factor)
    elif scaling == "yarn":
        def number(turns):                                   # of the pair that makes so many turns
            return half * math.log(original / (turns * 2 * math.pi)) / math.log(base)
        # (the end of the ramp may lie behind the last pair, which then keeps a part)
        first, last = max(math.floor(number(high)), 0), min(math.ceil(number(low)), rotary - 1)
        keep = 1.0 - ((pair - first) / max(last - first, 0.001)).clamp(0.0, 1.0)
        freqs = freqs * (keep + (1 - keep) / factor)
        scale = 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}; one of None, 'linear', 'ntk', 'wavelength', 'yarn'")
    return freqs.to(device), scale


class BatchPlan:
    """Where the newest tokens of a batch stand: table int32 [B, cols] of pages, kv_lens int32 [B]
    cached tokens with the new ones, cu_q int32 [B + 1] where each sequence's new tokens begin
    (None: one a sequence, its first B rows).  `tokens` is the number of rows of a step, with the padding before the
    first sequence and behind the last.  From them, on the GPU and without a copy to the host: positions and slots
    int64 [tokens] (slot -1: nothing is stored).  max_q, max_kv: see apex4.kv4_attention."""

    def __init__(self, table, kv_lens, cu_q=None, *, page: int, tokens: int | None = None, max_q: int | None = None,
                 max_kv: int | None = None):
        if page < 16 or page > 1024 or page & (page - 1):
            raise ValueError(f"page must be a power of two from 16 to 1024, got {page}")
        if table.dim() != 2 or table.shape[1] < 1:
            raise ValueError(f"table must be [B, cols] with a column at least, got {tuple(table.shape)}")
        B = table.shape[0]
        for name, t, shape in (("table", table, table.shape), ("kv_lens", kv_lens, (B,)), ("cu_q", cu_q, (B + 1,))):
            if t is not None and (t.dtype != torch.int32 or t.shape != shape or t.device != table.device):
                raise ValueError(f"{name} must be int32 {tuple(shape)} on {table.device}, "
                                 f"got {t.dtype} {tuple(t.shape)} on {t.device}")
        if tokens is not None and tokens < 0:
            raise ValueError(f"tokens must not be negative, got {tokens}")
        if tokens is None:
            if cu_q is not None:
                raise ValueError("tokens has to be given with cu_q (it is in device memory)")
            tokens = B
        if cu_q is None and tokens != B:
            if tokens < B:
                raise ValueError(f"{tokens} rows do not hold one token of each of {B} sequences")
            cu_q = torch.arange(B + 1, dtype=torch.int32, device=table.device)
            max_q = 1 if max_q is None else max_q
        self.positions, self.slots = self._places(table, kv_lens, cu_q, page, tokens)
        # (the attention takes them contiguous: parts of wider tables are copied)
        self.table, self.kv_lens = table.contiguous(), kv_lens.contiguous()
        self.cu_q = None if cu_q is None else cu_q.contiguous()
        self.page, self.tokens, self.max_q, self.max_kv = page, tokens, max_q, max_kv

    @staticmethod
    def _places(table, kv_lens, cu_q, page: int, tokens: int):
        B, cols = table.shape
        row = torch.arange(tokens, device=table.device)
        if B == 0:
            return torch.zeros_like(row), torch.full_like(row, -1)
        if cu_q is None:
            sequence, new = row, torch.ones_like(row)
        else:
            sequence = torch.searchsorted(cu_q[1:].long(), row, right=True)
            new = cu_q[1:].long()[sequence.clamp_max(B - 1)] - row
        owner = sequence.clamp_max(B - 1)
        position = kv_lens.long()[owner] - new
        live = (sequence < B) & (position >= 0) & (position < cols * page)
        if cu_q is not None:
            live &= row >= cu_q[0]
        held = position.clamp(0, cols * page - 1)
        at = table.long()[owner, held // page]
        return (torch.where(live, position, torch.zeros_like(position)),
                torch.where(live & (at >= 0), at * page + held % page, torch.full_like(position, -1)))


class KVCache4:
    """The paged 4-bit key/value cache of one layer: `pages` pages of `page` tokens for kv_heads
    heads of head_dim numbers (64, 128 or 256)."""

    def __init__(self, pages: int, kv_heads: int, head_dim: int, page: int = 64, device="cuda"):
        self.tensors = apex4.kv4_cache(pages, kv_heads, head_dim, page, device)
        self.pages, self.kv_heads, self.head_dim, self.page = pages, kv_heads, head_dim, page

    def _fits(self, plan: BatchPlan) -> None:
        if plan.page != self.page:
            raise ValueError(f"the plan is for pages of {plan.page} tokens, the cache has {self.page}")

    def append(self, k, v, plan: BatchPlan, inv_freq=None, q=None, **turn):
        """Stores the plan's tokens, turned by inv_freq where it is given; returns q turned."""
        self._fits(plan)
        positions = None if inv_freq is None else plan.positions
        return apex4.kv4_append(self.tensors, k, v, plan.slots, positions=positions, inv_freq=inv_freq, q=q, **turn)

    def attend(self, q, plan: BatchPlan, **args):
        """Attention of the plan's tokens over their sequences (apex4.kv4_attention's arguments)."""
        self._fits(plan)
        if q.shape[0] != plan.tokens:
            raise ValueError(f"q has {q.shape[0]} rows, the plan {plan.tokens}")
        return apex4.kv4_attention(q, self.tensors, plan.table, plan.kv_lens, plan.cu_q, max_q=plan.max_q,
                                   max_kv=plan.max_kv, **args)

    def read(self, slots, dtype=None):
        """(k, v) of the tokens at `slots` (apex4.kv4_read)."""
        return apex4.kv4_read(self.tensors, slots, dtype)


class CachedLayerW4A4(LlamaLayerW4A4):
    """One LLaMA-shaped decoder layer with attention over a 4-bit cache: the four W4A4 linears of
    `LlamaLayerW4A4`, and between QKV and O the rotation, the append and the attention.

    weights: as for LlamaLayerW4A4, "qkv" [(heads + 2 kv_heads) head_dim, h] and "o"
    [h, heads head_dim]; heads * head_dim need not be h.
    """

    def __init__(self, weights: dict, heads: int, kv_heads: int, head_dim: int, inv_freq, group: int = 128,
                 interleaved: bool = False, rope_scale: float = 1.0):
        super().__init__(weights, group)
        if weights["qkv"].shape[0] != (heads + 2 * kv_heads) * head_dim or weights["o"].shape[1] != heads * head_dim:
            raise ValueError(f"qkv {tuple(weights['qkv'].shape)} and o {tuple(weights['o'].shape)} do not fit "
                             f"{heads} and {kv_heads} heads of {head_dim}")
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.turn = dict(interleaved=interleaved, rope_scale=rope_scale)
        self.register_buffer("inv_freq", inv_freq)

    @classmethod
    def random(cls, hidden: int = 4096, intermediate: int = 11008, group: int = 128, seed: int = 0, device="cuda", *,
               heads: int = 32, kv_heads: int | None = None, head_dim: int = 128,
               base: float = 10000.0) -> "CachedLayerW4A4":
        """Random weights as LlamaLayerW4A4.random's, `kv_heads` key heads (as many as query heads when
        None), positions turned over the whole head."""
        kv_heads = heads if kv_heads is None else kv_heads
        shapes = {"qkv": ((heads + 2 * kv_heads) * head_dim, hidden), "o": (hidden, heads * head_dim),
                  "gate_up": (2 * intermediate, hidden), "down": (hidden, intermediate)}
        return cls(cls._random_weights(shapes, seed, device), heads, kv_heads, head_dim,
                   rope_frequencies(head_dim, base, device=device)[0], group)

    def forward(self, x: torch.Tensor, cache: KVCache4, plan: BatchPlan, window: int = 0) -> torch.Tensor:
        """x: fp16 [tokens, h], the plan's new tokens; their keys and values are added to the cache.
        Rows that no sequence owns come out as the layer's other parts make them (no attention)."""
        h, k = self.heads, self.kv_heads
        rows = self.qkv(x).view(x.shape[0], h + 2 * k, self.head_dim)
        q = cache.append(rows[:, h:h + k], rows[:, h + k:], plan, self.inv_freq, rows[:, :h], **self.turn)
        out = torch.zeros_like(q) if plan.cu_q is not None else None      # (rows behind the last sequence stay zero)
        o = cache.attend(q, plan, window=window, out=out)
        x = x + self.o(o.flatten(1))
        gu = self.gate_up(x)
        i = self.intermediate
        return x + self.down(torch.nn.functional.silu(gu[:, :i]) * gu[:, i:])
