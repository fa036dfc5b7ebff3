"""The 8-bit products where the matrix instruction cuts the most: in every run of
8 neighbouring k one product of the largest codes beside seven that are small
against it.  How far a sum may be off is in layers_ref.e4m3_gemm: at most 7 times
2^-13 of the largest product a run, beside the fp32 sums."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import layers_ref as ref  # noqa: E402
from w4a4_group_quantized_amd import apex4  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    apex4.lib()
    return torch.device("cuda:0")


def code_of(values):
    """E4M3 bytes of numbers that the format holds."""
    table = ref.e4m3_decode(np.arange(256))
    order = np.argsort(np.where(np.isnan(table), np.inf, table), kind="stable")[:254]
    at = order[np.searchsorted(table[order], values)]
    assert np.array_equal(table[at], values)
    return at.astype(np.uint8)


# small products just below and above the places that a sum beside 448 * 448 keeps
SMALL = [(2.0, 1.875), (2.0, 2.0), (3.75, 1.0), (3.75, 4.0), (5.0, 4.5), (7.5, 3.25), (15.0, 15.0)]


@pytest.mark.parametrize("M,N,K", [(3, 144, 1024), (16, 300, 4224), (40, 144, 512), (300, 136, 1408)])
@pytest.mark.parametrize("small", SMALL)
@pytest.mark.parametrize("cancel", [False, True])
def test_one_large_product_in_a_run(dev, M, N, K, small, cancel):
    rng = np.random.default_rng(M + K)
    a = np.full((M, K), small[0])
    w = np.full((N, K), small[1])
    large = 8 * np.arange(K // 8) + rng.integers(0, 8, K // 8)
    a[:, large] = 448.0
    # of one sign, or cancelling between the runs of a block
    w[:, large] = np.where(np.arange(K // 8) % 2, -448.0, 448.0) if cancel else 448.0
    sa = rng.uniform(0.5, 2.0, (M, K // 128)).astype(np.float32)
    sw = rng.uniform(0.5, 2.0, ((N + 127) // 128, K // 128)).astype(np.float32)
    args = [torch.from_numpy(t).to(dev) for t in (code_of(a), sa, code_of(w), sw)]
    _, y32 = apex4.gemm_e4m3(*args, torch.bfloat16, want_y32=True)
    want, bound = ref.e4m3_gemm(a, sa, w, sw)
    off = np.abs(y32.cpu().numpy().astype(np.float64) - want)
    assert np.all(off <= bound), float((off / bound).max())
