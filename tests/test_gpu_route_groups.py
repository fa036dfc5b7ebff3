"""apex4_route where the groups' scores are hard to tell apart in 32 bits: large
biases that cancel in a group's two best keys, mask values whose sum leaves the
fp32 range, equal keys.  ids equal to the plain implementation in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import layers_ref as ref  # noqa: E402
from w4a4_group_quantized_amd import apex4  # noqa: E402

pytestmark = pytest.mark.gpu
LOWEST = float(np.finfo(np.float32).min)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    apex4.lib()
    return torch.device("cuda:0")


def check(dev, logits, k, bias, **kw):
    ids, gates = apex4.route(torch.from_numpy(logits).to(dev), k, bias=torch.from_numpy(bias).to(dev), **kw)
    rid, rg = ref.route(logits, k, bias=bias, **kw)
    got = ids.cpu().numpy()
    wrong = np.argwhere((got != rid).any(1))[:, 0]
    assert wrong.size == 0, (wrong.size, got[wrong[0]], rid[wrong[0]])
    # one rounding to fp32 of 64-bit gates
    assert np.all(np.abs(gates.cpu().numpy() - rg) <= 2.0 ** -24 * (1 + 1e-6) * np.abs(rg) + 2.0 ** -149)


# experts, groups: 1, 4 and 16 values a lane
GROUPS = [(64, 32), (256, 64), (1024, 64)]


@pytest.mark.parametrize("E,n_group", GROUPS)
@pytest.mark.parametrize("size", [1e2, 1e3, 1e4])
@pytest.mark.parametrize("spread", [1.5, 1e-4])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("apart", [0.0, 0.03])
def test_biases_that_cancel_in_a_group(dev, E, n_group, size, spread, score, apart):
    """The two best keys of every group lie near +size and -size: their sums are
    about 1 and differ by as little as the spread of the scores.  `apart`: the
    groups' biases differ, so that their experts' keys are far from each other."""
    rng = np.random.default_rng(int(size) + E)
    M, per = 600, E // n_group
    logits = (spread * rng.standard_normal((M, E))).astype(np.float32)
    bias = np.full((n_group, per), -2 * size, dtype=np.float32)
    bias[:, 0] = size * (1 + apart * rng.permutation(n_group))
    bias[:, -1] = -bias[:, 0]
    bias[:, 1:-1] *= 1 + apart * n_group
    check(dev, logits, 8, bias.reshape(-1), score=score, n_group=n_group, topk_group=n_group // 2, group_top=2)


@pytest.mark.parametrize("E", [16, 256, 1024])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("top", [1, 2])
def test_lowest_biases_beside_a_dead_group(dev, E, score, top):
    """Two keys at the lowest fp32 number have a sum below it, which still is above a group without a live expert."""
    rng = np.random.default_rng(E)
    n_group, per = 4, E // 4
    logits = rng.standard_normal((40, E)).astype(np.float32)
    logits[:, per:2 * per] = -np.inf
    bias = np.zeros(E, dtype=np.float32)
    bias[2 * per:] = LOWEST
    k = min(64, per + 2)
    kw = dict(score=score, n_group=n_group, group_top=top)
    check(dev, logits, k, bias, topk_group=2, **kw)
    check(dev, logits, min(64, 2 * per), bias, topk_group=3, **kw)
    # dead group 0, and one live expert (so one key) in group 1
    logits = np.roll(logits, -per, axis=1)
    bias = np.full(E, LOWEST, dtype=np.float32)
    logits[:20, per + 1:2 * per] = -np.inf
    for keep in (1, 2, 3):
        check(dev, logits, min(64, keep * per), bias, topk_group=keep, **kw)


@pytest.mark.parametrize("E", [16, 256, 1024])
@pytest.mark.parametrize("top", [1, 2])
def test_highest_and_infinite_biases(dev, E, top):
    rng = np.random.default_rng(E)
    n_group, per = 4, E // 4
    logits = rng.standard_normal((40, E)).astype(np.float32)
    for value in (-LOWEST, np.inf):
        bias = np.zeros(E, dtype=np.float32)
        bias[per:per + 2] = value                  # sums beyond fp32
        bias[3 * per] = value
        bias[3 * per + 1] = LOWEST                 # a sum of 0 from the two ends
        for keep in (1, 2, 3):
            check(dev, logits, 8 if keep * per >= 8 else keep * per, bias, score="sigmoid", n_group=n_group,
                  topk_group=keep, group_top=top)


@pytest.mark.parametrize("E", [16, 256, 1024])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("n_group,top", [(1, 1), (4, 1), (4, 2)])
@pytest.mark.parametrize("base", [0.0, 100.0])
def test_equal_biased_keys(dev, E, score, n_group, top, base):
    """Equal keys, which 32 bits cannot tell apart: the lowest index wins, in experts and in groups."""
    rng = np.random.default_rng(E)
    logits = rng.integers(-1, 2, (30, E)).astype(np.float32)
    logits[0] = 0
    logits[1, ::2] = -np.inf
    bias = np.full(E, base, dtype=np.float32)
    check(dev, logits, 4, bias, score=score, n_group=n_group, topk_group=max(1, n_group // 2), group_top=top)
