"""apex4_rope against the rotation in 64 bits: within one rounding to fp32 and one to the type."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import attention_ref as ref  # noqa: E402
from w4a4_group_quantized_amd import apex4  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    apex4.lib()
    return torch.device("cuda:0")


def numbers(T, H, D, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, H, D), generator=g).to(getattr(torch, dtype))


def check(x, y, positions, freqs, dtype, interleaved=False, scale=1.0):
    want = ref.rope(x.double().cpu().numpy(), positions, freqs, interleaved, scale)
    # sines in fp64: 2^-46 of the pair; one rounding to fp32, one to the type
    bound = ref.rounding(want, dtype) + ref.rounding(want, "float32") + np.abs(want).max() * 2.0 ** -46
    over = np.abs(y.double().cpu().numpy() - want) > bound
    assert not over.any(), np.argwhere(over)[:4]


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("T,H,D,R,interleaved", [
    (1, 1, 16, 16, False), (1, 32, 128, 128, False), (3, 5, 64, 32, True), (65, 2, 80, 48, False), (7, 64, 128, 64, True),
    (2, 1, 256, 256, False), (33, 3, 96, 16, True), (300, 8, 64, 64, False), (1, 1024, 16, 16, True),
    (2, 3, 1024, 1024, False)])
def test_against_64_bits(dev, dtype, T, H, D, R, interleaved):
    x = numbers(T, H, D, dtype, T + H)
    positions = np.arange(T) * 37 + 5
    freqs = ref.frequencies(R, stretch=4.0 if interleaved else 1.0)
    y = apex4.rope(x.to(dev), torch.from_numpy(positions).to(dev), torch.from_numpy(freqs).to(dev),
                   interleaved=interleaved, scale=1.25)
    check(x, y, positions, freqs, dtype, interleaved, 1.25)
    if R < D:
        assert torch.equal(y[..., R:].cpu(), x[..., R:])


def test_far_and_odd_positions(dev):
    positions = np.array([0, 1, -1, -4097, 131071, 2 ** 20 + 1, 10 ** 6, 2 ** 31 - 1, -2 ** 31 + 1, 3, 3])
    x = numbers(len(positions), 4, 128, "float32", 3)
    freqs = ref.frequencies(128)
    y = apex4.rope(x.to(dev), torch.from_numpy(positions).to(dev), torch.from_numpy(freqs).to(dev))
    check(x, y, positions, freqs, "float32")
    assert torch.equal(y[0].cpu(), x[0])
    # beyond 32 bits a position is taken as the last
    far = torch.tensor([2 ** 31 - 1, 2 ** 40, -2 ** 31 + 1, -2 ** 62], device=dev)
    same = x[:1].expand(4, -1, -1).contiguous().to(dev)
    y = apex4.rope(same, far, torch.from_numpy(freqs).to(dev))
    assert torch.equal(y[0], y[1]) and torch.equal(y[2], y[3])


@pytest.mark.parametrize("interleaved", [False, True])
def test_parts_of_a_projection_and_in_place(dev, interleaved):
    """q and k as slices of one row of queries, keys and values; turned where they lie."""
    T, D, freqs = 9, 64, ref.frequencies(64)
    rows = numbers(T, 8, D, "bfloat16", 1).to(dev)
    positions = np.arange(T) + 100
    pos, freq = torch.from_numpy(positions).to(dev), torch.from_numpy(freqs).to(dev)
    before = rows.clone()
    q = apex4.rope(rows[:, :4], pos, freq, interleaved=interleaved)
    assert q.is_contiguous() and torch.equal(rows, before)
    check(before[:, :4], q, positions, freqs, "bfloat16", interleaved)
    assert apex4.rope(rows[:, 4:6], pos, freq, interleaved=interleaved, out=rows[:, 4:6]).data_ptr() == rows[:, 4:6].data_ptr()
    check(before[:, 4:6], rows[:, 4:6], positions, freqs, "bfloat16", interleaved)
    keep = [0, 1, 2, 3, 6, 7]
    assert torch.equal(rows[:, keep], before[:, keep])
    one = apex4.rope(rows[:1, :4], pos[:1], freq, interleaved=interleaved)
    assert torch.equal(one, q[:1])


def test_numbers_that_are_not_finite_stay_in_their_pair(dev):
    x = numbers(2, 2, 64, "float16").to(dev)
    clean = x.clone()
    x[0, 1, 3] = float("nan")
    x[1, 0, 40] = float("inf")
    pos, freq = torch.tensor([5, 6], device=dev), torch.from_numpy(ref.frequencies(64)).to(dev)
    y, want = apex4.rope(x, pos, freq), apex4.rope(clean, pos, freq)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[0, 1, [3, 35]] = True
    bad[1, 0, [8, 40]] = True
    assert torch.equal(y[~bad], want[~bad]) and not torch.isfinite(y[bad]).any()


def test_refusals(dev):
    x = torch.zeros((2, 2, 64), device=dev)
    pos, freq = torch.zeros(2, dtype=torch.int64, device=dev), torch.zeros(32, dtype=torch.float64, device=dev)
    with pytest.raises(ValueError):
        apex4.rope(x.cpu(), pos, freq)
    with pytest.raises(ValueError):
        apex4.rope(x.transpose(1, 2), pos, freq)
    with pytest.raises(ValueError):
        apex4.rope(x, pos.int(), freq)
    with pytest.raises(ValueError):
        apex4.rope(x, pos, freq.float())
    with pytest.raises(ValueError):
        apex4.rope(x, pos[:1], freq)
    with pytest.raises(ValueError):
        apex4.rope(x, None, freq)
    with pytest.raises(ValueError):
        apex4.rope(x, pos, freq, out=x.half())
    with pytest.raises(apex4.Apex4Error):
        apex4.rope(x, pos, torch.zeros(40, dtype=torch.float64, device=dev))
    assert apex4.rope(x[:0], pos[:0], freq).shape == (0, 2, 64)
