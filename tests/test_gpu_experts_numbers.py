"""apex4_experts_w4a4 with infinities and NaN: they show in the tokens they belong
to, and leave the other tokens' bits alone."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import layers_ref as ref  # noqa: E402
from w4a4_group_quantized_amd import apex4, inputs  # noqa: E402

pytestmark = pytest.mark.gpu
E, H, I = 6, 256, 384
VALUES = [float("nan"), float("inf"), -float("inf")]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    apex4.lib()
    return torch.device("cuda:0")


def problem(dev, M):
    """(x, ids, gates, weights): token m names experts m and m + 2 modulo 6, so that
    some tokens avoid expert 1 at every M."""
    rng = np.random.default_rng(M)
    w = []
    for n, k in ((2 * I, H), (H, I)):
        m = [ref.int4(inputs.weights(rng, n, k, 0.05)) for _ in range(E)]
        w.append(torch.from_numpy(np.stack([ref.pack(q) for q, _ in m])).to(dev))
        w.append(torch.from_numpy(np.stack([s for _, s in m])).to(dev))
    x = torch.from_numpy(rng.standard_normal((M, H), dtype=np.float32)).half().to(dev)
    at = torch.arange(M)
    ids = torch.stack([at % E, (at + 2) % E], 1).int().to(dev)
    return x, ids, torch.full((M, 2), 0.5, device=dev), w


# the two launches of a few tokens, and the tiles
TOKENS = [2, 12, 300]


@pytest.mark.parametrize("M", TOKENS)
@pytest.mark.parametrize("value", VALUES)
def test_a_tokens_own_values(dev, M, value):
    x, ids, gates, w = problem(dev, M)
    clean = apex4.experts(x, ids, gates, *w)
    assert torch.isfinite(clean).all()
    for column in (0, 131, H - 1):
        bad = x.clone()
        bad[M // 2, column] = value
        y, y32 = apex4.experts(bad, ids, gates, *w, want_y32=True)
        keep = torch.arange(M, device=dev) != M // 2
        assert torch.isnan(y[M // 2]).all() and torch.isnan(y32[M // 2]).all()
        assert torch.equal(y[keep], clean[keep])
        # without an expert nothing of the token counts
        none = ids.clone()
        none[M // 2] = -1
        y = apex4.experts(bad, none, gates, *w)
        assert (y[M // 2] == 0).all() and torch.isfinite(y).all()


@pytest.mark.parametrize("M", TOKENS)
@pytest.mark.parametrize("value", VALUES)
@pytest.mark.parametrize("row", [5, I + 5, None])
def test_scales_of_gate_and_up(dev, M, value, row):
    """One scale of a gate row or an up row, or all of the expert's."""
    x, ids, gates, w = problem(dev, M)
    clean = apex4.experts(x, ids, gates, *w)
    if row is None:
        w[1][1] = value
    else:
        w[1][1, row, 0] = value
    y = apex4.experts(x, ids, gates, *w)
    named = (ids == 1).any(1)
    assert named.any() and not named.all()
    assert torch.isnan(y[named]).all()
    assert torch.equal(y[~named], clean[~named])


@pytest.mark.parametrize("M", TOKENS)
@pytest.mark.parametrize("value", VALUES)
def test_scales_of_down(dev, M, value):
    x, ids, gates, w = problem(dev, M)
    clean = apex4.experts(x, ids, gates, *w)
    w[3][1, 7, 0] = value
    y = apex4.experts(x, ids, gates, *w)
    named = (ids == 1).any(1)
    assert named.any() and not named.all()
    assert not torch.isfinite(y[named, 7]).any()
    assert torch.equal(y[~named], clean[~named])
    rest = torch.arange(H, device=dev) != 7
    assert torch.equal(y[:, rest], clean[:, rest])
    w[3][1] = value
    y = apex4.experts(x, ids, gates, *w)
    assert not torch.isfinite(y[named]).any()
    assert torch.equal(y[~named], clean[~named])


@pytest.mark.parametrize("M", TOKENS)
def test_products_past_fp16_stay_within_it(dev, M):
    """Finite values only: h is kept within fp16 and nothing becomes infinite on the way."""
    x, ids, gates, w = problem(dev, M)
    w[1] *= 1000.0
    w[3] *= 1e-3
    y, y32 = apex4.experts(x, ids, gates, *w, want_y32=True)
    assert torch.isfinite(y).all() and torch.isfinite(y32).all()


@pytest.mark.parametrize("M", TOKENS)
@pytest.mark.parametrize("value", VALUES)
def test_zeros_times_what_is_no_number(dev, M, value):
    """A zero on one side of a product does not hide what is no number on the other."""
    x, ids, gates, w = problem(dev, M)
    named = (ids == 1).any(1)
    zeros = x.clone()
    zeros[:] = 0
    off = gates.clone()
    off[ids == 1] = 0
    clean, none = apex4.experts(x, ids, off, *w), apex4.experts(zeros, ids, gates, *w)
    broken = [t.clone() for t in w]
    broken[3][1] = value
    for y, other in ((apex4.experts(x, ids, off, *broken), clean), (apex4.experts(zeros, ids, gates, *broken), none)):
        assert not torch.isfinite(y[named]).any()
        assert torch.equal(y[~named], other[~named])
    off[ids == 1] = value
    y = apex4.experts(zeros, ids, off, *w)
    assert torch.isnan(y[named]).all() and (y[~named] == 0).all()


@pytest.mark.parametrize("M,experts,k,hidden,inter", [(2, 64, 8, 256, 1408), (3, 16, 4, 384, 2176), (4, 12, 5, 256, 1152),
                                                      (8, 6, 4, 128, 640), (16, 20, 2, 128, 640), (5, 3, 3, 256, 128),
                                                      (70, 12, 5, 256, 2176)])
def test_a_tokens_bits_go_by_its_own_slots(dev, M, experts, k, hidden, inter):
    """What the other tokens name, and what they hold, changes no bit of a token."""
    rng = np.random.default_rng(M + k)
    w = []
    for n, cols in ((2 * inter, hidden), (hidden, inter)):
        w.append(torch.from_numpy(rng.integers(0, 256, (experts, n, cols // 2), dtype=np.uint8)).to(dev))
        w.append(torch.from_numpy(rng.uniform(0.001, 0.01, (experts, n, cols // 128)).astype(np.float32)).to(dev))
    x = torch.from_numpy(rng.standard_normal((M, hidden), dtype=np.float32)).half().to(dev)
    gates = torch.from_numpy(rng.uniform(-1.0, 1.0, (M, k)).astype(np.float32)).to(dev)
    ids = rng.integers(-1, experts, (M, k)).astype(np.int32)
    ids[0] = rng.permutation(experts)[:k]
    _, first = apex4.experts(x, torch.from_numpy(ids).to(dev), gates, *w, want_y32=True)
    for m in (0, M // 2, M - 1):
        for draw in range(6):
            other = rng.integers(-1, experts, (M, k)).astype(np.int32)
            if draw == 5:
                other[:] = -1
            other[m] = ids[m]
            z = torch.from_numpy(rng.standard_normal((M, hidden), dtype=np.float32)).half().to(dev)
            z[m] = x[m]
            _, y32 = apex4.experts(z, torch.from_numpy(other).to(dev), gates, *w, want_y32=True)
            assert torch.equal(y32[m], first[m]), (m, draw)
