"""E4M3Linear, W4A4Experts and SparseLayerW4A4 (w4a4_group_quantized_amd/sparse.py):
the modules give the library calls' bits, and router and experts together the
plain implementation's values."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import layers_ref as ref  # noqa: E402
from w4a4_group_quantized_amd import apex4, inputs  # noqa: E402
from w4a4_group_quantized_amd.sparse import E4M3Linear, SparseLayerW4A4, W4A4Experts  # noqa: E402

E, H, I, K = 16, 256, 128, 4


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    apex4.lib()
    return torch.device("cuda:0")


def layer_of(dev, shared, seed=0):
    rng = np.random.default_rng(seed)
    gu = np.stack([inputs.weights(rng, 2 * I, H, 0.05) for _ in range(E)])
    down = np.stack([inputs.weights(rng, H, I, 0.05) for _ in range(E)])
    router = torch.from_numpy(rng.standard_normal((E, H), dtype=np.float32) * 0.1).to(dev)
    bias = torch.from_numpy(0.1 * rng.standard_normal(E).astype(np.float32)).to(dev)
    ex = W4A4Experts.from_weights(torch.from_numpy(gu).to(dev), torch.from_numpy(down).to(dev))
    pair = None
    if shared:
        pair = [E4M3Linear.from_weight(torch.from_numpy(inputs.weights(rng, n, k, 0.05)).to(dev))
                for n, k in ((2 * I, H), (H, I))]
    layer = SparseLayerW4A4(router, ex, K, pair, score="sigmoid", bias=bias, n_group=4, topk_group=2, group_top=2,
                            scale=2.5)
    return layer, gu, down


def tokens(dev, M, seed):
    return torch.from_numpy(inputs.activations(np.random.default_rng(seed), M, H, "outlier", seed)).to(dev)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 3, 50, 300])
def test_layer_against_the_plain_one(dev, M):
    layer, gu, down = layer_of(dev, shared=False)
    x = tokens(dev, M, M)
    padding = torch.arange(M, device=dev) >= max(1, M - M // 4)
    y = layer(x, padding)
    ids, gates = layer.route(x, padding)
    torch.cuda.synchronize()
    logits = torch.nn.functional.linear(x.float(), layer.router).masked_fill(padding.unsqueeze(1), float("-inf"))
    rid, _ = ref.route(logits.cpu().numpy(), K, "sigmoid", layer.bias.cpu().numpy(), 4, 2, 2, True, 2.5)
    assert np.array_equal(ids.cpu().numpy(), rid)
    want, bound = ref.experts(x.cpu().numpy(), rid, gates.cpu().numpy(), [ref.int4(w) for w in gu],
                              [ref.int4(w) for w in down])
    # y is the fp16 rounding: half a unit of fp16 (2^-11, and 2^-25 of a subnormal) beside the bound
    got = y.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - want) <= bound + (np.abs(want) + bound) * 2.0 ** -11 + 2.0 ** -25)
    assert (got[padding.cpu().numpy()] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [2, 40])
def test_modules_give_the_calls_bits(dev, M):
    layer, _, _ = layer_of(dev, shared=True)
    ex = layer.experts
    x = tokens(dev, M, 7)
    ids, gates = layer.route(x)
    y = apex4.experts(x, ids, gates, ex.qw_gate_up, ex.s_gate_up, ex.qw_down, ex.s_down)
    g, u = apex4.linear_e4m3(x, layer.shared[0].qw8, layer.shared[0].sw).chunk(2, dim=-1)
    s = apex4.linear_e4m3((torch.nn.functional.silu(g) * u).contiguous(), layer.shared[1].qw8, layer.shared[1].sw)
    assert torch.equal(layer(x), y + s)
    # leading dimensions and rows with a stride
    wide = torch.zeros((M, 2 * H), dtype=torch.float16, device=dev)
    wide[:, ::2] = x
    assert torch.equal(layer(wide[:, ::2]), y + s)
    assert torch.equal(layer(x.view(2, M // 2, H)), (y + s).view(2, M // 2, H))
    lin = layer.shared[0]
    assert torch.equal(lin(x.view(2, M // 2, H)).view(M, -1), lin(x))
    assert lin(x.bfloat16()).dtype == torch.bfloat16


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 24])
def test_layer_graph_replays(dev, M):
    layer, _, _ = layer_of(dev, shared=True)
    x = tokens(dev, M, 1)
    layer(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer(x)
    for seed in range(4):
        x.copy_(tokens(dev, M, 30 + seed))
        graph.replay()
        torch.cuda.synchronize()
        want = layer(x)                      # eager work between the replays
        torch.cuda.synchronize()
        assert torch.equal(y, want), seed


@pytest.mark.gpu
def test_two_streams_at_once(dev):
    """Calls that overlap on two streams, each with its own workspace."""
    layer, _, _ = layer_of(dev, shared=True)
    xs = [tokens(dev, m, m) for m in (1, 130)]
    want = [layer(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(layer(xs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


@pytest.mark.gpu
def test_module_refusals_on_the_gpu(dev):
    layer, _, _ = layer_of(dev, shared=True)
    x = tokens(dev, 4, 1)
    with pytest.raises(ValueError):
        layer(x[:, :128])
    with pytest.raises(ValueError):
        layer.experts(x, torch.zeros((4, 2), dtype=torch.int64, device=dev), torch.zeros((4, 2), device=dev))
    with pytest.raises(ValueError):
        layer.shared[0](x.float())
    with pytest.raises(ValueError):
        SparseLayerW4A4(layer.router[:, :128], layer.experts, K)
    with pytest.raises(apex4.Apex4Error):
        apex4.route(torch.zeros((2, 8), device=dev), 9)
    with pytest.raises(ValueError):
        apex4.route(torch.zeros((2, 8), device=dev), 2, score="argmax")
    small = torch.empty(16, dtype=torch.uint8, device=dev)
    ids, gates = layer.route(x)
    ex = layer.experts
    with pytest.raises(apex4.Apex4Error):
        apex4.experts(x, ids, gates, ex.qw_gate_up, ex.s_gate_up, ex.qw_down, ex.s_down, workspace=small)


def test_modules_refuse_host_tensors():
    with pytest.raises(ValueError):
        E4M3Linear(torch.zeros((8, 128), dtype=torch.uint8), torch.ones((1, 1)))
    z = torch.zeros((2, 256, 64), dtype=torch.uint8)
    with pytest.raises(ValueError):
        W4A4Experts(z, z, z, z)
