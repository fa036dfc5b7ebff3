"""The ends of what the routing, expert and 8-bit calls allow: values that are
no numbers beside ones that are, an expert named twice, outputs at any address,
sizes whose offsets pass 32 bits, graphs that share a workspace."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import layers_ref as ref  # noqa: E402
from w4a4_group_quantized_amd import apex4, inputs  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    apex4.lib()
    return torch.device("cuda:0")


def normal(shape, seed, dtype=torch.float16):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape, dtype=np.float32)).to(dtype)


def experts_on(dev, E, H, I, seed=0):
    rng = np.random.default_rng(seed)
    gu = [ref.int4(inputs.weights(rng, 2 * I, H, 0.05)) for _ in range(E)]
    down = [ref.int4(inputs.weights(rng, H, I, 0.05)) for _ in range(E)]
    w = []
    for m in (gu, down):
        w.append(torch.from_numpy(np.stack([ref.pack(q) for q, _ in m])).to(dev))
        w.append(torch.from_numpy(np.stack([s for _, s in m])).to(dev))
    return w, gu, down


@pytest.mark.parametrize("M", [2, 12, 300])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_e4m3_keeps_what_is_no_number_to_its_row(dev, M, value):
    N, K = 200, 1280
    x, w = normal((M, K), 1).to(dev), normal((N, K), 2).to(dev)
    x[:, 256:384] = 0                        # a block whose scale is 0 without the value
    qw, sw = apex4.pack_weight_e4m3(w)
    clean = apex4.linear_e4m3(x, qw, sw)
    for column in (3, 300):
        bad = x.clone()
        bad[M // 2, column] = value
        y = apex4.linear_e4m3(bad, qw, sw)
        assert torch.isnan(y[M // 2]).all()
        keep = torch.arange(M, device=dev) != M // 2
        assert torch.equal(y[keep], clean[keep])
        qa, sa = apex4.quantize_e4m3(bad)
        assert torch.equal(apex4.gemm_e4m3(qa, sa, qw, sw)[keep], clean[keep])
    w[7, 5] = float("nan")                   # a weight: its output column
    qn, sn = apex4.pack_weight_e4m3(w)
    y = apex4.linear_e4m3(x, qn, sn)
    assert torch.isnan(y[:, 7]).all() and not torch.isnan(y[:, 8:]).any()


@pytest.mark.parametrize("M", [2, 12, 300])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_experts_keep_what_is_no_number_to_its_tokens(dev, M, value):
    E, H, I, k = 6, 256, 384, 2
    w, _, _ = experts_on(dev, E, H, I)
    x = normal((M, H), 3).to(dev)
    ids = torch.stack([torch.arange(M) % E, (torch.arange(M) + 1) % E], 1).int().to(dev)
    gates = torch.full((M, k), 0.5, device=dev)
    clean = apex4.experts(x, ids, gates, *w)
    bad = x.clone()
    bad[0, 9] = value
    assert torch.equal(apex4.experts(bad, ids, gates, *w)[1:], clean[1:])
    # an expert whose scales are no numbers, and gates of a token that are none
    broken = [t.clone() for t in w]
    broken[1][1] = value
    broken[3][1] = value
    others = ~(ids == 1).any(1)
    if others.any():
        assert torch.equal(apex4.experts(x, ids, gates, *broken)[others], clean[others])
    ids2, gates2 = ids.clone(), gates.clone()
    ids2[0, 1] = 1                           # the broken expert beside a whole one
    gates2[M - 1] = value
    y = apex4.experts(x, ids2, gates2, *w)
    assert torch.equal(y[1:M - 1], clean[1:M - 1]) and not torch.isfinite(y[M - 1]).any()
    # places without an expert, whatever their gate
    ids2[:, 1] = -1
    gates2.copy_(gates)
    want = apex4.experts(x, ids2, gates2, *w)
    gates2[:, 1] = value
    assert torch.equal(apex4.experts(x, ids2, gates2, *w), want)


@pytest.mark.parametrize("M", [2, 5])
def test_few_tokens_beside_a_broken_expert(dev, M):
    """Token 0 names experts 0 and 1, the others 2 and 3; expert 1's scales are infinite."""
    w, _, _ = experts_on(dev, 4, 256, 256)
    x = normal((M, 256), 3).to(dev)
    ids = torch.full((M, 2), 2, dtype=torch.int32, device=dev)
    ids[:, 1] = 3
    ids[0] = torch.tensor([0, 1], dtype=torch.int32)
    gates = torch.full((M, 2), 0.5, device=dev)
    clean = apex4.experts(x, ids, gates, *w)
    w[3][1] = float("inf")
    assert torch.equal(apex4.experts(x, ids, gates, *w)[1:], clean[1:])


@pytest.mark.parametrize("M", [1, 6, 100])
def test_the_same_expert_several_times(dev, M):
    E, H, I, k = 3, 256, 256, 5
    w, gu, down = experts_on(dev, E, H, I, 4)
    x = inputs.activations(np.random.default_rng(M), M, H, "outlier", M)
    ids = np.tile(np.array([2, 0, 2, 2, 0], dtype=np.int32), (M, 1))
    ids[M // 2] = 1
    gates = np.random.default_rng(9).uniform(-1.0, 1.0, (M, k)).astype(np.float32)
    y, y32 = apex4.experts(torch.from_numpy(x).to(dev), torch.from_numpy(ids).to(dev), torch.from_numpy(gates).to(dev),
                           *w, want_y32=True)
    want, bound = ref.experts(x, ids, gates, gu, down)
    assert np.all(np.abs(y32.cpu().numpy().astype(np.float64) - want) <= bound)
    assert torch.equal(y, y32.half())


@pytest.mark.parametrize("M,E,k,H,I", [(40, 2, 1, 128, 2048), (70, 3, 3, 256, 2176), (20, 4, 2, 384, 4096)])
def test_experts_whose_down_products_run_in_parts(dev, M, E, k, H, I):
    w, gu, down = experts_on(dev, E, H, I, 6)
    x = inputs.activations(np.random.default_rng(M), M, H, "outlier", M)
    rng = np.random.default_rng(9)
    ids = rng.integers(-1, E + 1, (M, k)).astype(np.int32)
    gates = rng.uniform(-1.0, 1.0, (M, k)).astype(np.float32)
    args = [torch.from_numpy(t).to(dev) for t in (x, ids, gates)]
    y, y32 = apex4.experts(*args, *w, want_y32=True)
    want, bound = ref.experts(x, ids, gates, gu, down)
    assert np.all(np.abs(y32.cpu().numpy().astype(np.float64) - want) <= bound)
    assert torch.equal(y, y32.half()) and torch.equal(apex4.experts(*args, *w), y)


@pytest.mark.parametrize("M", [2, 20, 300])
@pytest.mark.parametrize("N", [64, 129])
def test_e4m3_outputs_at_any_address(dev, M, N):
    K = 640
    x, w = normal((M, K), 1).to(dev), normal((N, K), 2).to(dev)
    qw, sw = apex4.pack_weight_e4m3(w)
    want, want32 = apex4.linear_e4m3(x, qw, sw, want_y32=True)
    y = torch.full((M * N + 2,), 7.0, dtype=torch.float16, device=dev)
    y32 = torch.full((M * N + 2,), 7.0, device=dev)
    apex4.linear_e4m3(x, qw, sw, want_y32=True, y=y[1:-1].view(M, N), y32=y32[1:-1].view(M, N))
    assert torch.equal(y[1:-1].view(M, N), want) and torch.equal(y32[1:-1].view(M, N), want32)
    assert (y[[0, -1]] == 7).all() and (y32[[0, -1]] == 7).all()


def test_route_of_the_most_rows(dev):
    M = 2 ** 25
    logits = torch.randint(-3, 4, (M, 2), device=dev, dtype=torch.int8).half()
    ids, gates = apex4.route(logits, 1, renormalize=False, score="sigmoid")
    want = (logits[:, 1] > logits[:, 0])
    assert torch.equal(ids[:, 0], want.int())
    p = torch.sigmoid(logits.float().max(1).values)
    # two fp32 sigmoids, each within a few roundings of its value below 1
    assert float((gates[:, 0] - p).abs().max()) < 2.0 ** -21


@pytest.mark.parametrize("E", [8, 200])
def test_route_bias_of_minus_infinity_masks_the_choice_only(dev, E):
    logits = normal((9, E), 5, torch.float32)
    bias = torch.zeros(E)
    bias[::2] = -float("inf")
    bias[1] = float("nan")
    ids, gates = apex4.route(logits.to(dev), 4, bias=bias.to(dev), renormalize=False)
    rid, rg = ref.route(logits.numpy(), 4, "softmax", bias.numpy(), renormalize=False)
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert np.allclose(gates.cpu().numpy(), rg, rtol=2.0 ** -23, atol=0)   # 64 bits, one rounding


def test_experts_with_offsets_past_32_bits(dev):
    """2^24 slots: the rows between the products lie past 2^31 values and 2^33 bytes."""
    period, M, k, E, H = 64, (1 << 18) + 64, 64, 4, 128
    w, _, _ = experts_on(dev, E, H, H)
    x = normal((period, H), 1).to(dev)
    ids = torch.randint(0, E, (period, k), device=dev, dtype=torch.int32)
    gates = torch.rand((period, k), device=dev) / 8
    few = apex4.experts(x, ids, gates, *w)
    y = apex4.experts(x.repeat(M // period, 1), ids.repeat(M // period, 1), gates.repeat(M // period, 1), *w)
    # one group of K in both products and slots added in their order: the same bits at every place
    assert torch.equal(y.view(-1, period, H), few.expand(M // period, period, H))


@pytest.mark.parametrize("M,N,K", [(262208, 16, 16512), (131136, 16400, 128)])
def test_e4m3_with_offsets_past_32_bits(dev, M, N, K):
    """x of more than 2^32 values; y of more than 2^31."""
    period = 64
    x, w = normal((period, K), 1).to(dev), normal((N, K), 2).to(dev)
    qw, sw = apex4.pack_weight_e4m3(w)
    qa, sa = apex4.quantize_e4m3(x)
    y = apex4.linear_e4m3(x.repeat(M // period, 1), qw, sw).view(-1, period, N)
    want, bound = ref.e4m3_gemm(ref.e4m3_decode(qa.cpu().numpy()), sa.cpu().numpy(),
                                ref.e4m3_decode(qw.cpu().numpy()), sw.cpu().numpy())
    # y is the fp16 rounding: half a unit beside the bound of the fp32 sum
    bound = bound + (np.abs(want) + bound) * 2.0 ** -11 + 2.0 ** -25
    low, high = (torch.from_numpy(v).to(dev) for v in (want - bound, want + bound))
    for part in y.split(64):
        d = part.double()
        assert bool(((d >= low) & (d <= high)).all())


def test_graphs_that_share_a_workspace(dev):
    """Two captured layers with one workspace, replayed in turn on one stream."""
    w, _, _ = experts_on(dev, 4, 256, 256)
    q8, s8 = apex4.pack_weight_e4m3(normal((256, 4096), 2).to(dev))
    sizes = [(1, 2), (70, 2)]
    ws = torch.empty(max([apex4.experts_workspace_size(m, k, 4, 256, 256) for m, k in sizes] +
                         [apex4.linear_e4m3_workspace_size(m, 256, 4096) for m, _ in sizes]),
                     dtype=torch.uint8, device=dev)
    runs = []
    for i, (m, k) in enumerate(sizes):
        x, z = normal((m, 256), i).to(dev), normal((m, 4096), 10 + i).to(dev)
        ids, gates = apex4.route(normal((m, 4), 20 + i).to(dev), k)

        def call(x=x, z=z, ids=ids, gates=gates, ws=None):
            return apex4.experts(x, ids, gates, *w, workspace=ws), apex4.linear_e4m3(z, q8, s8, workspace=ws)

        want = call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call(ws=ws)
        runs.append((graph, got, want, call))   # (call holds the inputs, which the graph reads)
    for _ in range(4):
        for graph, got, *_ in runs:
            for t in got:
                t.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for _, got, want, _ in runs:
            assert all(torch.equal(g, v) for g, v in zip(got, want))
