"""Layers on several streams at once: no call shares a workspace with another."""
import pytest

torch = pytest.importorskip("torch")

from w4a4_group_quantized_amd import apex4  # noqa: E402
from w4a4_group_quantized_amd.attention import BatchPlan, CachedLayerW4A4, KVCache4, rope_frequencies  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    apex4.lib()
    return torch.device("cuda:0")


@pytest.mark.parametrize("tokens", [1, 40])
def test_one_layer_on_two_streams(dev, tokens):
    """Two batches of equal row counts through one layer, each with a cache of its own; and a captured
    step replayed beside an eager one."""
    h, i, heads, kv, D = 512, 768, 8, 4, 64
    g = torch.Generator().manual_seed(2)
    shapes = {"qkv": ((heads + 2 * kv) * D, h), "o": (h, heads * D), "gate_up": (2 * i, h), "down": (h, i)}
    w = {n: (0.05 * torch.randn(s, generator=g)).half().to(dev) for n, s in shapes.items()}
    m = CachedLayerW4A4(w, heads, kv, D, rope_frequencies(D, device=dev)[0])
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    plan = BatchPlan(i32([[0, 1, 2]]), i32([tokens]), i32([0, tokens]), page=16, tokens=tokens, max_q=tokens, max_kv=48)
    xs = [torch.randn((tokens, h), generator=g).half().to(dev) for _ in range(2)]
    caches = [KVCache4(3, kv, D, 16, dev) for _ in range(2)]
    want = [m(x, c, plan) for x, c in zip(xs, caches)]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(m(xs[k], caches[k], plan))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[k]) for k in range(2) for y in got[k])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        y = m(xs[0], caches[0], plan)
    for _ in range(5):
        with torch.cuda.stream(streams[0]):
            graph.replay()
        with torch.cuda.stream(streams[1]):
            other = m(xs[1], caches[1], plan)
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(other, want[1])
