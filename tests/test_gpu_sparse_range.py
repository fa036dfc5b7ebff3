"""The shared expert of SparseLayerW4A4 where its values leave the range of fp16."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from w4a4_group_quantized_amd import apex4, inputs  # noqa: E402
from w4a4_group_quantized_amd.sparse import E4M3Linear, SparseLayerW4A4, W4A4Experts  # noqa: E402

pytestmark = pytest.mark.gpu
E, H, I = 4, 256, 128


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    apex4.lib()
    return torch.device("cuda:0")


def layer_of(dev, gate, up):
    """Every gate row and every up row of the shared expert holds one value; its down rows hold 2^-10."""
    rng = np.random.default_rng(0)
    ex = W4A4Experts.from_weights(*(torch.from_numpy(np.stack([inputs.weights(rng, n, k, 0.05) for _ in range(E)]))
                                    .to(dev) for n, k in ((2 * I, H), (H, I))))
    first = torch.cat([torch.full((I, H), gate), torch.full((I, H), up)]).half().to(dev)
    shared = [E4M3Linear.from_weight(first), E4M3Linear.from_weight(torch.full((H, I), 2.0 ** -10).half().to(dev))]
    router = torch.from_numpy(rng.standard_normal((E, H), dtype=np.float32)).to(dev)
    return SparseLayerW4A4(router, ex, 2, shared)


# x = 1 in every column: gate and up are 256 times their weights, exactly
@pytest.mark.parametrize("M", [1, 20])
@pytest.mark.parametrize("gate,up,h", [(1.0, 1.0, 65504.0), (1.0, -2.0, -65504.0), (300.0, 1.0, 65504.0),
                                       (-300.0, 1.0, 0.0), (-300.0, 300.0, 0.0), (0.5, 300.0, 65504.0),
                                       (0.25, 0.5, 8192.0)])
def test_products_beyond_the_type(dev, M, gate, up, h):
    layer = layer_of(dev, gate, up)
    x = torch.ones((M, H), dtype=torch.float16, device=dev)
    ids, gates = layer.route(x)
    y = layer(x) - layer.experts(x, ids, gates)
    # 128 equal values of h, whose code is 448: 128 h 2^-10, and the roundings of fp16 sums near the experts' part
    want = 128 * h * 2.0 ** -10
    e = layer.experts(x, ids, gates).float().abs().max().item()
    assert torch.isfinite(y).all()
    # the scales h / 448 and 2^-10 / 448 are rounded (2^-24 each, and their product), the linear layer's output,
    # the sum and the difference to fp16 (2^-11 each)
    assert (y.float() - want).abs().max().item() <= 3 * 2.0 ** -11 * (abs(want) + 2 * e) + 4 * 2.0 ** -24 * abs(want)


def test_what_is_no_number_stays(dev):
    layer = layer_of(dev, 1.0, 1.0)
    x = torch.ones((3, H), dtype=torch.float16, device=dev)
    x[1, 5] = float("nan")
    y = layer(x)
    assert torch.isnan(y[1]).all() and torch.isfinite(y[[0, 2]]).all()
