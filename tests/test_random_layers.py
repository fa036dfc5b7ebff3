"""Layers with random weights (on the CPU: packing is replaced)."""
import pytest

torch = pytest.importorskip("torch")

from w4a4_group_quantized_amd.attention import CachedLayerW4A4, rope_frequencies  # noqa: E402
from w4a4_group_quantized_amd.linear import LlamaLayerW4A4, W4A4Linear  # noqa: E402


class Packed(torch.nn.Module):
    def __init__(self, w, group):
        super().__init__()
        self.w, self.group = w, group


@pytest.fixture(autouse=True)
def packing(monkeypatch):
    monkeypatch.setattr(W4A4Linear, "from_weight", classmethod(lambda cls, w, group=128, group_a=None: Packed(w, group)))


def weights(layer):
    return {n: getattr(layer, n).w for n in LlamaLayerW4A4.NAMES}


def test_random_layer_with_attention():
    m = CachedLayerW4A4.random(64, 96, 32, 3, "cpu", heads=4, kv_heads=2, head_dim=64, base=500.0)
    assert {n: tuple(w.shape) for n, w in weights(m).items()} == {"qkv": (512, 64), "o": (64, 256), "gate_up": (192, 64),
                                                                 "down": (64, 96)}
    assert (m.heads, m.kv_heads, m.head_dim, m.hidden, m.intermediate, m.qkv.group) == (4, 2, 64, 64, 96, 32)
    assert torch.equal(m.inv_freq, rope_frequencies(64, 500.0, device="cpu")[0])
    again = CachedLayerW4A4.random(64, 96, 32, 3, "cpu", heads=4, kv_heads=2, head_dim=64)
    other = CachedLayerW4A4.random(64, 96, 32, 4, "cpu", heads=4, kv_heads=2, head_dim=64)
    assert all(torch.equal(a, b) for a, b in zip(weights(m).values(), weights(again).values()))
    assert not torch.equal(m.o.w, other.o.w)
    assert tuple(CachedLayerW4A4.random(64, 96, seed=1, device="cpu", heads=2, head_dim=64).qkv.w.shape) == (384, 64)


def test_random_layer_without():
    m = LlamaLayerW4A4.random(64, 96, 32, 3, "cpu")
    assert tuple(m.qkv.w.shape) == (192, 64) and tuple(m.o.w.shape) == (64, 64) and m.qkv.group == 32
