"""Frequencies of rotary positions for longer contexts, against their definitions (CPU)."""
import math

import pytest

torch = pytest.importorskip("torch")

from w4a4_group_quantized_amd.attention import BatchPlan, rope_frequencies  # noqa: E402


def plain(rotary, base=10000.0):
    return torch.tensor([base ** (-2.0 * i / rotary) for i in range(rotary // 2)], dtype=torch.float64)


def test_scalings():
    f, s = rope_frequencies(128, device="cpu")
    assert f.dtype == torch.float64 and torch.allclose(f, plain(128), rtol=1e-14) and s == 1.0
    f, s = rope_frequencies(64, 500000.0, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(f, plain(64, 500000.0) / 4, rtol=1e-14) and s == 1.0
    f, _ = rope_frequencies(128, scaling="ntk", factor=8.0, device="cpu")
    p = plain(128)
    assert f[0] == 1.0 and math.isclose(f[-1], p[-1] / 8, rel_tol=1e-12) and (f <= p * (1 + 1e-14)).all()


def test_wavelength_scaling():
    f, s = rope_frequencies(128, 500000.0, scaling="wavelength", factor=8.0, original=8192, low=1.0, high=4.0,
                            device="cpu")
    p = plain(128, 500000.0)
    wave = 2 * math.pi / p
    slow, fast = wave > 8192 / 1.0, wave < 8192 / 4.0
    assert torch.allclose(f[slow], p[slow] / 8, rtol=1e-14) and torch.allclose(f[fast], p[fast], rtol=1e-14)
    mid = ~slow & ~fast
    smooth = (8192 / wave[mid] - 1.0) / 3.0
    assert mid.any() and torch.allclose(f[mid], (1 - smooth) * p[mid] / 8 + smooth * p[mid], rtol=1e-13) and s == 1.0


def test_yarn_scaling():
    f, s = rope_frequencies(128, scaling="yarn", factor=16.0, original=4096, low=1.0, high=32.0, device="cpu")
    p = plain(128)
    # pairs that make 32 and 1 turns in 4096 positions: 128 ln(4096 / (2 pi n)) / (2 ln 10000)
    first, last = 20, 46
    assert math.floor(64 * math.log(4096 / (64 * math.pi)) / math.log(10000)) == first
    assert math.ceil(64 * math.log(4096 / (2 * math.pi)) / math.log(10000)) == last
    assert torch.allclose(f[:first + 1], p[:first + 1], rtol=1e-14)
    assert torch.allclose(f[last:], p[last:] / 16, rtol=1e-14)
    keep = 1 - (33 - first) / (last - first)
    assert math.isclose(f[33], p[33] * (keep + (1 - keep) / 16), rel_tol=1e-13)
    assert math.isclose(s, 0.1 * math.log(16.0) + 1.0)
    assert rope_frequencies(64, scaling="yarn", device="cpu")[1] == 1.0


def test_refusals():
    for bad in (dict(rotary=24), dict(rotary=0), dict(rotary=64, factor=0.5), dict(rotary=64, scaling="other")):
        with pytest.raises(ValueError):
            rope_frequencies(device="cpu", **bad)


def test_plan():
    """Two sequences and two rows of padding: the first's 3 newest of 5 tokens, the second's 1 of 18."""
    table = torch.tensor([[4, -1], [2, 7]], dtype=torch.int32)
    plan = BatchPlan(table, torch.tensor([5, 18], dtype=torch.int32), torch.tensor([0, 3, 4], dtype=torch.int32),
                     page=16, tokens=6)
    assert plan.positions.tolist() == [2, 3, 4, 17, 0, 0]
    assert plan.slots.tolist() == [66, 67, 68, 7 * 16 + 1, -1, -1]
    plan = BatchPlan(table, torch.tensor([0, 33], dtype=torch.int32), page=16)     # an empty place; one token too many
    assert plan.slots.tolist() == [-1, -1] and plan.positions.tolist() == [0, 0]
    plan = BatchPlan(table, torch.tensor([17, 1], dtype=torch.int32), page=16)     # a page that is none
    assert plan.slots.tolist() == [-1, 32] and plan.positions.tolist() == [16, 0]
    with pytest.raises(ValueError):
        BatchPlan(table, torch.tensor([1, 1], dtype=torch.int32), torch.tensor([0, 1, 2], dtype=torch.int32), page=16)
