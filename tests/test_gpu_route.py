"""apex4_route against a plain implementation in 64 bits: ids equal, gates
within the rounding to fp32 (half a unit, 2^-24, and a hair for the 64-bit
arithmetic on both sides)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import layers_ref as ref  # noqa: E402
from w4a4_group_quantized_amd import apex4  # noqa: E402

pytestmark = pytest.mark.gpu
RTOL = 2.0 ** -24 * (1 + 1e-6)
TINY = 2.0 ** -149          # half a unit of a subnormal fp32 number, and then some


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    apex4.lib()
    return torch.device("cuda:0")


def check(dev, logits, k, bias=None, **kw):
    """logits: a CPU tensor of the type under test."""
    b = None if bias is None else torch.from_numpy(bias).to(dev)
    ids, gates = apex4.route(logits.to(dev), k, bias=b, **kw)
    torch.cuda.synchronize()
    rid, rg = ref.route(logits.double().numpy(), k, bias=bias, **kw)
    got_i, got_g = ids.cpu().numpy(), gates.cpu().numpy().astype(np.float64)
    assert np.array_equal(got_i, rid), np.argwhere(got_i != rid)[:5]
    assert np.all(np.abs(got_g - rg) <= RTOL * np.abs(rg) + TINY)
    assert np.all(got_g[rid < 0] == 0)
    return ids, gates


def logits_of(M, E, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (1.5 * torch.randn((M, E), generator=g)).to(dtype)


SHAPES = [(1, 1, 1), (1, 64, 6), (5, 7, 7), (3, 65, 64), (17, 96, 4), (9, 160, 6), (64, 256, 8), (2, 257, 3),
          (6, 512, 10), (3, 1000, 22), (2, 1024, 64)]


@pytest.mark.parametrize("M,E,k", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_plain_top_k(dev, M, E, k, score, renormalize):
    check(dev, logits_of(M, E, M + E), k, score=score, renormalize=renormalize)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_half_types_with_many_ties(dev, dtype, score):
    # 1000 draws of bf16 or fp16 numbers hold many equal ones: the lowest index wins
    check(dev, logits_of(11, 1000, 3, dtype), 40, score=score)
    check(dev, torch.zeros((3, 130), dtype=dtype), 9, score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("E,n_group,keep,k", [(8, 2, 1, 3), (160, 8, 3, 6), (256, 8, 4, 8), (60, 60, 7, 7),
                                              (64, 64, 9, 9), (1024, 32, 5, 20), (90, 3, 2, 60)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_groups(dev, score, top, E, n_group, keep, k, with_bias):
    rng = np.random.default_rng(E + n_group)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32) if with_bias else None
    check(dev, logits_of(13, E, E + k), k, bias=bias, score=score, n_group=n_group, topk_group=keep, group_top=top,
          scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_bias_ranks_but_does_not_weigh(dev, score):
    bias = np.zeros(32, dtype=np.float32)
    bias[[3, 30]] = 5.0
    ids, _ = check(dev, logits_of(8, 32, 1), 4, bias=bias, score=score, renormalize=False)
    assert set(ids[:, :2].flatten().tolist()) == {3, 30}
    bias[30] = -np.inf
    ids, _ = check(dev, logits_of(8, 32, 1), 31, bias=bias, score=score)
    assert not (ids == 30).any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("n_group,top", [(1, 1), (4, 1), (4, 2)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_masked_experts_and_empty_rows(dev, score, with_bias, n_group, top, renormalize):
    E, k = 64, 6
    x = logits_of(8, E, 9)
    x[0] = -np.inf                       # padding
    x[1, 1:] = -np.inf                   # one live expert
    x[2] = torch.finfo(torch.float32).min
    x[3, 5:] = torch.finfo(torch.float32).min
    x[4, ::2] = float("nan")
    x[5, 16:] = float("nan")             # three groups without a live expert
    x[6, 7] = np.inf
    bias = np.linspace(-0.05, 0.05, E).astype(np.float32) if with_bias else None
    ids, gates = check(dev, x, k, bias=bias, score=score, n_group=n_group, topk_group=max(1, n_group // 2),
                       group_top=top, renormalize=renormalize)
    assert (ids[0] == -1).all() and (gates[0] == 0).all()
    assert ids[1].tolist() == [0] + [-1] * (k - 1)
    assert torch.isfinite(gates).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_far_scores(dev, score):
    """Scores that underflow in 32 bits, and a large logit in a group that is not kept."""
    x = torch.full((4, 16), -200.0)
    x[0] += torch.arange(16) * 0.25
    x[1, 0] = 300.0
    x[2] = torch.linspace(-700, 700, 16)
    x[3] = torch.linspace(20, 60, 16)    # sigmoids that are 1 in 32 bits
    check(dev, x, 5, score=score)
    check(dev, x, 5, score=score, renormalize=False)
    # group 0's best is the one large logit; with sums of two the others win
    check(dev, x, 4, score=score, n_group=4, topk_group=2, group_top=2)


def test_out_buffers_streams_and_empty(dev):
    x = logits_of(33, 64, 4).to(dev)
    ref_i, ref_g = apex4.route(x, 8)
    ids = torch.full((35, 8), 77, dtype=torch.int32, device=dev)
    gates = torch.full((35, 8), 77.0, device=dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        apex4.route(x, 8, out=(ids[1:34], gates[1:34]))
    torch.cuda.synchronize()
    assert torch.equal(ids[1:34], ref_i) and torch.equal(gates[1:34], ref_g)
    assert (ids[[0, 34]] == 77).all() and (gates[[0, 34]] == 77).all()      # rows beside the call's
    ids, gates = apex4.route(x[:0], 8)
    assert ids.shape == (0, 8) and gates.shape == (0, 8)


def test_graph_replays(dev):
    x = logits_of(100, 256, 5).to(dev)
    bias = torch.zeros(256, device=dev)
    kw = dict(score="sigmoid", bias=bias, n_group=8, topk_group=4, group_top=2)
    apex4.route(x, 8, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ids, gates = apex4.route(x, 8, **kw)
    for seed in range(4):
        x.copy_(logits_of(100, 256, 50 + seed))
        graph.replay()
        torch.cuda.synchronize()
        want = apex4.route(x, 8, **kw)
        torch.cuda.synchronize()
        assert torch.equal(ids, want[0]) and torch.equal(gates, want[1])
