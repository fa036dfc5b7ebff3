"""The 8-bit block-scaled calls (apex4_quantize_e4m3, apex4_pack_weight_e4m3,
apex4_gemm_e4m3, apex4_linear_e4m3) against a plain implementation in 64 bits:
codes and scales equal, products within the bound of fp32 sums, y the rounding
of y32."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import layers_ref as ref  # noqa: E402
from w4a4_group_quantized_amd import apex4  # noqa: E402

pytestmark = pytest.mark.gpu
HALVES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    apex4.lib()
    return torch.device("cuda:0")


def acts(M, K, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g)
    x[:, torch.randperm(K, generator=g)[:max(1, K // 100)]] *= 20
    return x.to(dtype)


def weights(N, K, seed, dtype):
    g = torch.Generator().manual_seed(1000 + seed)
    return (0.02 * torch.randn((N, K), generator=g)).to(dtype)


def same_codes(q8, s, x, rows):
    want, ws = ref.e4m3_quantize(x.float().numpy(), rows)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), ws.view(np.uint32))
    assert np.array_equal(ref.e4m3_decode(q8.cpu().numpy()), want)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("rows,K", [(1, 128), (3, 256), (129, 384), (260, 1024)])
def test_quantizers_equal_the_rule(dev, dtype, rows, K):
    x = acts(rows, K, rows + K, dtype)
    x[0, :128] = 0                                       # a block of zeros
    x[-1, -128:] = torch.linspace(-1, 1, 128).to(dtype)  # every binade of the codes
    same_codes(*apex4.quantize_e4m3(x.to(dev)), x, 1)
    same_codes(*apex4.pack_weight_e4m3(x.to(dev)), x, 128)


@pytest.mark.parametrize("dtype", HALVES)
def test_quantizer_ties_and_extremes(dev, dtype):
    """Quotients halfway between two codes (a maximum of 448 makes the scale 1),
    subnormal codes, the smallest and largest numbers of the type."""
    row = torch.zeros(128)
    row[0] = 448
    halves = [17, 19, 21, 23, 25, 27, 29, 31, 8.5, 9.5, 2.0 ** -10, 3 * 2.0 ** -10, 5 * 2.0 ** -10, 2.0 ** -11,
              2.0 ** -7 + 2.0 ** -10, 432, 416, 400]
    row[1:1 + len(halves)] = torch.tensor(halves)
    row[40:40 + len(halves)] = -torch.tensor(halves)
    x = torch.zeros((6, 128))
    x[0] = row
    x[1] = row * 2.0 ** -8
    fin = torch.finfo(dtype)
    x[2, :4] = torch.tensor([fin.max, -fin.max, fin.max / 2, 1.0])
    x[3, :4] = torch.tensor([fin.smallest_normal, -fin.smallest_normal / 2, fin.smallest_normal / 4, 0.0])
    x[4, :3] = torch.tensor([-0.0, 0.0, -0.0])
    x[5, :3] = torch.tensor([2.0 ** -24, -2.0 ** -24, 2.0 ** -24])   # the smallest fp16 number
    x = x.to(dtype)
    same_codes(*apex4.quantize_e4m3(x.to(dev)), x, 1)


def check_gemm(dev, M, N, K, seed, dtype):
    x, w = acts(M, K, seed, dtype), weights(N, K, seed, dtype)
    qa, sa = apex4.quantize_e4m3(x.to(dev))
    qw, sw = apex4.pack_weight_e4m3(w.to(dev))
    y = torch.full((M + 2, N), 7.0, dtype=dtype, device=dev)
    y32 = torch.full((M + 2, N), 7.0, device=dev)
    apex4.gemm_e4m3(qa, sa, qw, sw, dtype, want_y32=True, y=y[1:-1], y32=y32[1:-1])
    lin, lin32 = apex4.linear_e4m3(x.to(dev), qw, sw, want_y32=True)
    torch.cuda.synchronize()
    want, bound = ref.e4m3_gemm(ref.e4m3_decode(qa.cpu().numpy()), sa.cpu().numpy(),
                                ref.e4m3_decode(qw.cpu().numpy()), sw.cpu().numpy())
    got = y32[1:-1].cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - want) <= bound), float((np.abs(got - want) / np.maximum(bound, 1e-300)).max())
    assert torch.equal(y[1:-1], y32[1:-1].to(dtype))
    assert (y[[0, -1]] == 7).all() and (y32[[0, -1]] == 7).all()       # rows beside the call's
    assert torch.equal(lin32, y32[1:-1]) and torch.equal(lin, y[1:-1])  # the linear call gives the same bits


# one row to several tiles of rows; columns and rows that end inside a tile or
# a block of 128; one block of K, and numbers of blocks that fill no item
SHAPES = [(1, 1, 128), (4, 33, 4096), (5, 200, 4096), (16, 40, 1024), (1, 48, 16384), (1, 128, 128), (2, 17, 256), (3, 130, 640), (16, 96, 512), (17, 257, 384), (33, 64, 1152),
          (64, 384, 1024), (65, 129, 896), (128, 128, 128), (130, 300, 768), (257, 520, 640), (300, 1000, 256),
          (513, 136, 1408),
          (9, 9000, 4224), (16, 70000, 640), (24, 8300, 5248), (3, 300, 114816)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", HALVES)
def test_products(dev, M, N, K, dtype):
    check_gemm(dev, M, N, K, M + N, dtype)


@pytest.mark.parametrize("M,N,K", [(5, 48, 11008), (70, 40, 28672), (300, 264, 8192)])
def test_long_sums(dev, M, N, K):
    check_gemm(dev, M, N, K, 5, torch.bfloat16)


@pytest.mark.parametrize("M", [3, 300])
def test_codes_at_the_ends(dev, M):
    """Products of the largest codes, of one sign: sums that no cancelling helps."""
    N, K = 144, 512
    qa = torch.full((M, K), 0x7E, dtype=torch.uint8, device=dev)     # 448
    qw = torch.full((N, K), 0xFE, dtype=torch.uint8, device=dev)     # -448
    sa = torch.full((M, K // 128), 2.0 ** -9, device=dev)
    sw = torch.full((2, K // 128), 2.0 ** -9, device=dev)
    sw[1] = 2.0 ** -8
    y, y32 = apex4.gemm_e4m3(qa, sa, qw, sw, torch.bfloat16, want_y32=True)
    torch.cuda.synchronize()
    want = -448.0 * 448.0 * K * 2.0 ** -18
    assert (y32[:, :128] == want).all() and (y32[:, 128:] == 2 * want).all()


@pytest.mark.parametrize("M", [1, 40, 300])
def test_graph_stream_and_repeat(dev, M):
    N, K = 520, 1024
    w = weights(N, K, 3, torch.float16).to(dev)
    qw, sw = apex4.pack_weight_e4m3(w)
    x = acts(M, K, 1, torch.float16).to(dev)
    first = apex4.linear_e4m3(x, qw, sw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = apex4.linear_e4m3(x, qw, sw)
    torch.cuda.synchronize()
    assert torch.equal(first, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = apex4.linear_e4m3(x, qw, sw)
    for seed in range(4):
        x.copy_(acts(M, K, 20 + seed, torch.float16))
        graph.replay()
        torch.cuda.synchronize()
        want = apex4.linear_e4m3(x, qw, sw)
        torch.cuda.synchronize()
        assert torch.equal(y, want), seed


def test_empty(dev):
    qw, sw = apex4.pack_weight_e4m3(weights(64, 256, 0, torch.float16).to(dev))
    x = torch.empty((0, 256), dtype=torch.float16, device=dev)
    assert apex4.linear_e4m3(x, qw, sw).shape == (0, 64)
    q, s = apex4.quantize_e4m3(x)
    assert q.shape == (0, 256) and s.shape == (0, 2)
    assert apex4.gemm_e4m3(q, s, qw, sw).shape == (0, 64)
