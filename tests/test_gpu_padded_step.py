"""Steps of a padded batch through the layer with attention."""
import pytest

torch = pytest.importorskip("torch")

from w4a4_group_quantized_amd import apex4  # noqa: E402
from w4a4_group_quantized_amd.attention import BatchPlan, CachedLayerW4A4, KVCache4  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    apex4.lib()
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def layer(dev):
    return CachedLayerW4A4.random(256, 384, 128, 1, dev, heads=4, kv_heads=2, head_dim=64)


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def test_decoding_with_rows_behind_the_batch(dev, layer):
    """Three sequences in a step of eight rows: as the three alone (other row counts take other linear
    kernels, with the same codes and sums)."""
    table, lens = i32([[0, 1], [2, 3], [4, 5]], dev), i32([3, 20, 1], dev)
    x = torch.randn((8, 256), generator=torch.Generator().manual_seed(1)).half().to(dev)
    caches = [KVCache4(6, 2, 64, 16, dev) for _ in range(2)]
    y = layer(x, caches[0], BatchPlan(table, lens, page=16, tokens=8))
    want = layer(x[:3], caches[1], BatchPlan(table, lens, page=16))
    assert y.shape == (8, 256) and torch.isfinite(y).all()
    for a, b in zip(caches[0].tensors, caches[1].tensors):
        assert torch.equal(a, b)
    # (fp32 sums in another order: at most a step of fp16 and of a code of the next linear's input)
    assert ((y[:3] - want).float().norm(dim=-1) <= 0.1 * want.float().norm(dim=-1)).all()


def test_step_without_sequences(dev, layer):
    """Rows of padding only: nothing is stored, every row comes out."""
    cache = KVCache4(2, 2, 64, 16, dev)
    none = torch.zeros((0, 3), dtype=torch.int32, device=dev)
    x = torch.randn((4, 256), generator=torch.Generator().manual_seed(2)).half().to(dev)
    y = layer(x, cache, BatchPlan(none, i32([], dev), page=16, tokens=4))
    assert torch.isfinite(y).all() and all((t == 0).all() for t in cache.tensors)


def test_step_without_rows(dev, layer):
    cache = KVCache4(2, 2, 64, 16, dev)
    x = torch.zeros((0, 256), dtype=torch.float16, device=dev)
    assert layer(x, cache, BatchPlan(torch.zeros((0, 3), dtype=torch.int32, device=dev), i32([], dev), page=16)).shape == x.shape
    plan = BatchPlan(i32([[0, 1]], dev), i32([3], dev), i32([0, 0], dev), page=16, tokens=0)
    assert layer(x, cache, plan).shape == x.shape and all((t == 0).all() for t in cache.tensors)
