"""Sparse expert layers on the library's calls, and linear layers kept in 8 bits.

`E4M3Linear` is a linear layer in 8-bit floating point with a scale for each
block of 128 (apex4_linear_e4m3), for the layers of a W4A4 model that 4 bits
cost too much.  `W4A4Experts` holds the packed INT4 weights of a sparse
layer's experts and runs them over routed tokens (apex4_experts_w4a4).
`SparseLayerW4A4` is the layer: the router's projection (a plain matrix
product), apex4_route, the experts, and where there is one the shared expert
that every token passes, in 8 bits.

The modules keep no workspace: every call takes its own from torch's caching
allocator, so calls on different streams do not share one.
"""
from __future__ import annotations

import torch

from . import apex4


def _rows(x: torch.Tensor, features: int) -> torch.Tensor:
    if x.shape[-1] != features:
        raise ValueError(f"expected [..., {features}] input, got {tuple(x.shape)}")
    return x.reshape(-1, features).contiguous()


class E4M3Linear(torch.nn.Module):
    """y = x W^T with W held as E4M3 bytes and one fp32 scale per 128 x 128 block.

    qw8: uint8 [N, K], sw: float32 [ceil(N/128), K/128] (apex4_pack_weight_e4m3
    outputs).  Inputs: fp16 or bf16 [..., K] on the GPU; the output has their type.
    """

    def __init__(self, qw8: torch.Tensor, sw: torch.Tensor):
        super().__init__()
        if qw8.dtype != torch.uint8 or qw8.dim() != 2 or not qw8.is_cuda:
            raise ValueError("qw8 must be a uint8 [N, K] GPU tensor (apex4_pack_weight_e4m3 output)")
        self.out_features, self.in_features = qw8.shape
        self.register_buffer("qw8", qw8)
        self.register_buffer("sw", sw)

    @classmethod
    def from_weight(cls, w: torch.Tensor) -> "E4M3Linear":
        """Quantize an fp16 or bf16 [N, K] GPU weight (the offline step)."""
        return cls(*apex4.pack_weight_e4m3(w.contiguous()))

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        y = apex4.linear_e4m3(_rows(x, self.in_features), self.qw8, self.sw)
        return y.reshape(*x.shape[:-1], self.out_features)

    def extra_repr(self) -> str:
        return f"in_features={self.in_features}, out_features={self.out_features}"


class W4A4Experts(torch.nn.Module):
    """The experts of a sparse layer: down(silu(gate x) * up x) of each, W4A4 with groups of 128.

    qw_gate_up: uint8 [E, 2I, H/2] (the I gate rows first), s_gate_up: float32
    [E, 2I, H/128], qw_down: uint8 [E, H, I/2], s_down: float32 [E, H, I/128].
    """

    def __init__(self, qw_gate_up, s_gate_up, qw_down, s_down):
        super().__init__()
        for name, t in (("qw_gate_up", qw_gate_up), ("qw_down", qw_down)):
            if t.dtype != torch.uint8 or t.dim() != 3 or not t.is_cuda:
                raise ValueError(f"{name} must be a uint8 [E, rows, bytes] GPU tensor (apex4_pack_weight output)")
        self.experts, self.hidden = qw_down.shape[:2]
        self.intermediate = 2 * qw_down.shape[2]
        for name, t in (("qw_gate_up", qw_gate_up), ("s_gate_up", s_gate_up), ("qw_down", qw_down),
                        ("s_down", s_down)):
            self.register_buffer(name, t)

    @classmethod
    def from_weights(cls, gate_up: torch.Tensor, down: torch.Tensor) -> "W4A4Experts":
        """Quantize and pack fp16 [E, 2I, H] and [E, H, I] GPU weights (the offline step)."""
        packed = []
        for w in (gate_up, down):
            with torch.cuda.device(w.device):      # (the library launches to the current device)
                q, s = apex4.pack_weight(w.reshape(-1, w.shape[-1]).contiguous(), 128)
            packed += [q.view(*w.shape[:2], -1), s.view(*w.shape[:2], -1)]
        return cls(*packed)

    def forward(self, x: torch.Tensor, ids: torch.Tensor, gates: torch.Tensor) -> torch.Tensor:
        """x: fp16 [..., H]; ids int32, gates float32 [tokens, k] (apex4.route): ids outside the
        experts add nothing."""
        y = apex4.experts(_rows(x, self.hidden), ids, gates, self.qw_gate_up, self.s_gate_up, self.qw_down,
                          self.s_down)
        return y.reshape(x.shape)

    def extra_repr(self) -> str:
        return f"experts={self.experts}, hidden={self.hidden}, intermediate={self.intermediate}"


class SparseLayerW4A4(torch.nn.Module):
    """Router, experts and (optionally) a shared expert of one sparse feed-forward layer.

    router: [E, H] weight of the router's projection, in the type the logits are
    to be computed in; experts: W4A4Experts; shared: (gate_up, down) as
    E4M3Linear, applied to every token; routing: keyword arguments of
    apex4.route (score, bias, n_group, topk_group, group_top, renormalize, scale).
    A token whose logits are all NaN (a NaN in x) is routed nowhere, like padding:
    only the shared expert shows it.
    """

    def __init__(self, router: torch.Tensor, experts: W4A4Experts, k: int, shared=None, **routing):
        super().__init__()
        if tuple(router.shape) != (experts.experts, experts.hidden):
            raise ValueError(f"router must be {(experts.experts, experts.hidden)}, got {tuple(router.shape)}")
        self.k = k
        self.experts = experts
        self.shared = None if shared is None else torch.nn.ModuleList(shared)
        self.register_buffer("router", router)
        self.register_buffer("bias", routing.pop("bias", None))
        self.routing = routing

    def route(self, x: torch.Tensor, padding: torch.Tensor | None = None):
        """(ids, gates) of the tokens x [tokens, H]; `padding`: bool [tokens], True for tokens
        that are routed nowhere."""
        logits = torch.nn.functional.linear(x.to(self.router.dtype), self.router)
        if padding is not None:
            logits = logits.masked_fill(padding.unsqueeze(1), float("-inf"))
        return apex4.route(logits, self.k, bias=self.bias, **self.routing)

    def forward(self, x: torch.Tensor, padding: torch.Tensor | None = None) -> torch.Tensor:
        rows = _rows(x, self.experts.hidden)
        ids, gates = self.route(rows, None if padding is None else padding.reshape(-1))
        y = self.experts(rows, ids, gates)
        if self.shared is not None:
            # within the type's range, as the routed experts' h: an infinity would cost the token its whole row
            # (the codes of a block with one are NaN), and silu(-inf) is NaN; a NaN stays
            most = torch.finfo(rows.dtype).max
            gate, up = self.shared[0](rows).clamp_(-most, most).chunk(2, dim=-1)
            y = y + self.shared[1]((torch.nn.functional.silu(gate) * up).clamp_(-most, most))
        return y.reshape(x.shape)
