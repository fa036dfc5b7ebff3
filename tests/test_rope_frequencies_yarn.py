"""YaRN's frequencies over the whole range of contexts, by its definition (CPU)."""
import math

import pytest

torch = pytest.importorskip("torch")

from w4a4_group_quantized_amd.attention import rope_frequencies  # noqa: E402


def yarn(rotary, base, factor, original, low, high):
    """Pair d turns original * base^(-2 d / rotary) / (2 pi) times; the numbers d that make `high` and
    `low` turns, rounded outwards and kept within 0 .. rotary - 1, bound the ramp (the upper one may lie
    behind the last pair)."""
    def number(turns):
        return rotary * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
    first, last = max(math.floor(number(high)), 0), min(math.ceil(number(low)), rotary - 1)
    out = []
    for d in range(rotary // 2):
        f = base ** (-2.0 * d / rotary)
        ramp = min(max((d - first) / (last - first if last != first else 0.001), 0.0), 1.0)
        out.append(f / factor * ramp + f * (1 - ramp))
    return torch.tensor(out, dtype=torch.float64), number


@pytest.mark.parametrize("rotary,base", [(128, 10000.0), (64, 10000.0), (128, 1e6), (32, 500.0)])
@pytest.mark.parametrize("original", [2048, 4096, 32768, 65536, 131072, 10 ** 6])
def test_yarn_over_contexts(rotary, base, original):
    f, _ = rope_frequencies(rotary, base, scaling="yarn", factor=8.0, original=original, low=1.0, high=32.0, device="cpu")
    want, number = yarn(rotary, base, 8.0, original, 1.0, 32.0)
    assert torch.allclose(f, want, rtol=1e-13)
    plain = rope_frequencies(rotary, base, device="cpu")[0]
    if number(1.0) > rotary / 2 - 1:                         # every pair makes more than `low` turns
        assert (f > plain / 8 * 1.0001).all()


def test_yarn_by_default_blends_from_32_turns_to_1():
    want = yarn(128, 10000.0, 4.0, 4096, 1.0, 32.0)[0]
    assert torch.allclose(rope_frequencies(128, scaling="yarn", factor=4.0, device="cpu")[0], want, rtol=1e-13)
    by_wavelength = rope_frequencies(128, scaling="wavelength", factor=4.0, device="cpu")[0]       # as before: from 4
    assert torch.equal(by_wavelength, rope_frequencies(128, scaling="wavelength", factor=4.0, high=4.0, device="cpu")[0])


def test_refusals():
    for scaling in ("wavelength", "yarn"):
        for bad in (dict(low=4.0, high=4.0), dict(low=4.0, high=1.0), dict(low=0.0), dict(low=-1.0), dict(original=0)):
            with pytest.raises(ValueError):
                rope_frequencies(128, scaling=scaling, factor=2.0, device="cpu", **bad)
    for base in (1.0, 0.0, -10.0, float("nan")):
        with pytest.raises(ValueError):
            rope_frequencies(128, base, scaling="yarn", factor=2.0, device="cpu")
