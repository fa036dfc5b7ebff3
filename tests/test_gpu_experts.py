"""apex4_experts_w4a4 against a plain implementation in 64 bits (layers_ref.experts,
which also says how far a right fp32 computation may be from it)."""
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


def make(E, H, I, seed):
    """(codes, scales) of every expert's two matrices, on the host."""
    rng = np.random.default_rng(seed)
    gu = [ref.int4(inputs.weights(rng, 2 * I, H, 0.05)) for _ in range(E)]
    down = [ref.int4(inputs.weights(rng, H, I, 0.05)) for _ in range(E)]
    return gu, down


def to_gpu(dev, gu, down):
    out = []
    for m in (gu, down):
        out.append(torch.from_numpy(np.stack([ref.pack(q) for q, _ in m])).to(dev))
        out.append(torch.from_numpy(np.stack([s for _, s in m])).to(dev))
    return out


def check(dev, x, ids, gates, gu, down):
    M, H = x.shape
    w = to_gpu(dev, gu, down)
    y = torch.full((M + 2, H), 7.0, dtype=torch.float16, device=dev)
    y32 = torch.full((M + 2, H), 7.0, device=dev)
    args = (torch.from_numpy(x).to(dev), torch.from_numpy(ids).to(dev), torch.from_numpy(gates).to(dev))
    apex4.experts(*args, *w, want_y32=True, y16=y[1:-1], y32=y32[1:-1])
    again = apex4.experts(*args, *w)
    torch.cuda.synchronize()
    want, bound = ref.experts(x, ids, gates, gu, down)
    got = y32[1:-1].cpu().numpy().astype(np.float64)
    over = np.abs(got - want) > bound
    assert not over.any(), (np.argwhere(over)[:4], np.abs(got - want).max(), bound[over][:4])
    assert torch.equal(y[1:-1], y32[1:-1].half())
    assert torch.equal(again, y[1:-1])
    assert (y[[0, -1]] == 7).all() and (y32[[0, -1]] == 7).all()        # rows beside the call's
    return got, want


def tokens(M, H, seed):
    return inputs.activations(np.random.default_rng(seed), M, H, "outlier", seed)


def spread(M, E, k, seed):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(M)]).astype(np.int32).reshape(M, k)
    gates = rng.uniform(0.05, 1.0, (M, k)).astype(np.float32)
    return ids, gates


SHAPES = [  # M, E, k, H, I
    (1, 1, 1, 128, 128), (1, 8, 2, 256, 128), (1, 64, 8, 128, 256), (2, 3, 3, 640, 384), (7, 5, 2, 1152, 128),
    (17, 4, 1, 256, 640), (40, 4, 2, 384, 256), (33, 2, 2, 128, 1152), (70, 2, 1, 256, 256), (150, 3, 2, 512, 128),
    (200, 70, 4, 128, 128), (300, 4, 2, 256, 384), (600, 3, 2, 128, 256)]


@pytest.mark.parametrize("M,E,k,H,I", SHAPES)
def test_against_64_bits(dev, M, E, k, H, I):
    gu, down = make(E, H, I, E + I)
    check(dev, tokens(M, H, M), *spread(M, E, k, M + E), gu, down)


@pytest.mark.parametrize("M", [5, 90, 400])
def test_all_tokens_to_one_expert(dev, M):
    E, H, I = 6, 256, 256
    gu, down = make(E, H, I, 2)
    ids = np.full((M, 1), 4, dtype=np.int32)
    gates = np.linspace(0.1, 1, M).astype(np.float32).reshape(M, 1)
    check(dev, tokens(M, H, 3), ids, gates, gu, down)


@pytest.mark.parametrize("M", [6, 120, 500])
def test_places_without_an_expert(dev, M):
    """Ids outside [0, E), padding tokens, an expert named twice; the gates of
    dead places are NaN and infinity and enter nothing."""
    E, H, I, k = 5, 256, 128, 3
    gu, down = make(E, H, I, 7)
    ids, gates = spread(M, E, k, 8)
    ids[1::3, 0] = -1
    ids[2::5, 1] = E
    ids[3::7, 2] = 2 ** 31 - 1
    ids[4::5, 1] = -2 ** 31
    ids[0] = 3                                    # the same expert in every place
    ids[M // 2:] = -1                             # padding
    dead = (ids < 0) | (ids >= E)
    gates[dead] = np.where(np.arange(dead.sum()) % 2, np.nan, np.inf)
    x = tokens(M, H, 9)
    got, _ = check(dev, x, ids, gates, gu, down)
    assert (got[M // 2:] == 0).all()
    # nothing live at all
    got, _ = check(dev, x, np.full_like(ids, -1), gates, gu, down)
    assert (got == 0).all()


def test_zero_rows_and_large_products(dev):
    """A token of zeros, a zero matrix, and products beyond fp16 that are kept within it."""
    E, H, I = 3, 256, 128
    gu, down = make(E, H, I, 4)
    gu[1] = (gu[1][0], gu[1][1] * np.float32(3000))
    gu[2] = (gu[2][0] * 0, gu[2][1])
    x = tokens(9, H, 5)
    x[4] = 0
    ids, gates = spread(9, E, 2, 6)
    got, _ = check(dev, x, ids, gates, gu, down)
    assert np.isfinite(got).all() and (got[4] == 0).all()


@pytest.mark.parametrize("M", [1, 3, 40, 400])
def test_graph_stream_and_workspace(dev, M):
    E, H, I, k = 8, 256, 256, 2
    w = to_gpu(dev, *make(E, H, I, 11))
    x = torch.from_numpy(tokens(M, H, 1)).to(dev)
    ids, gates = (torch.from_numpy(a).to(dev) for a in spread(M, E, k, 1))
    need = apex4.experts_workspace_size(M, k, E, H, I)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=dev)      # NaN patterns
    first = apex4.experts(x, ids, gates, *w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = apex4.experts(x, ids, gates, *w, workspace=ws[:need])
    torch.cuda.synchronize()
    assert torch.equal(first, other)
    assert (ws[need:] == 255).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = apex4.experts(x, ids, gates, *w, workspace=ws[:need])
    for seed in range(5):
        x.copy_(torch.from_numpy(tokens(M, H, 20 + seed)))
        n_ids, n_gates = spread(M, E, k, 30 + seed)
        if seed == 3:
            n_ids[:] = -1
        ids.copy_(torch.from_numpy(n_ids))
        gates.copy_(torch.from_numpy(n_gates))
        graph.replay()
        torch.cuda.synchronize()
        want = apex4.experts(x, ids, gates, *w)
        torch.cuda.synchronize()
        assert torch.equal(y, want), seed


def test_empty(dev):
    w = to_gpu(dev, *make(2, 128, 128, 0))
    y = apex4.experts(torch.empty((0, 128), dtype=torch.float16, device=dev),
                      torch.empty((0, 2), dtype=torch.int32, device=dev), torch.empty((0, 2), device=dev), *w)
    assert y.shape == (0, 128)


def test_routed_layer(dev):
    """Router and experts as they are used together: padding rows of the
    router's logits come out as zeros, the others as the plain layer's."""
    M, E, k, H, I = 50, 16, 4, 256, 128
    gu, down = make(E, H, I, 21)
    w = to_gpu(dev, gu, down)
    x = tokens(M, H, 22)
    logits = torch.from_numpy(np.random.default_rng(23).standard_normal((M, E)).astype(np.float32))
    logits[40:] = -np.inf
    ids, gates = apex4.route(logits.to(dev), k, score="sigmoid", n_group=4, topk_group=2, group_top=2, scale=2.5)
    y, y32 = apex4.experts(torch.from_numpy(x).to(dev), ids, gates, *w, want_y32=True)
    torch.cuda.synchronize()
    rid, _ = ref.route(logits.numpy(), k, "sigmoid", None, 4, 2, 2, True, 2.5)
    assert np.array_equal(ids.cpu().numpy(), rid)
    want, bound = ref.experts(x, rid, gates.cpu().numpy(), gu, down)
    assert np.all(np.abs(y32.cpu().numpy() - want) <= bound)
    assert (y[40:] == 0).all()
