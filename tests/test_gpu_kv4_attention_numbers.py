"""apex4_kv4_attention where the numbers are far apart, against single rows in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import attention_ref as ref  # noqa: E402
from attention_rows import attention_rows, cut  # noqa: E402
from w4a4_group_quantized_amd import apex4  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    apex4.lib()
    return torch.device("cuda:0")


def run(dev, q, host, table, lens, cu, **args):
    to = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(dev)  # noqa: E731
    cache = tuple(torch.from_numpy(a).to(dev) for a in host.arrays())
    o, lse = apex4.kv4_attention(q.to(dev), cache, to(table), to(lens), None if cu is None else to(cu), want_lse=True,
                                 **args)
    torch.cuda.synchronize()
    return o.double().cpu().numpy(), lse.double().cpu().numpy()


def close(got, got_lse, want, dtype, rows):
    o, lse, bound, lse_bound = want
    for at, (t, h) in enumerate(rows):
        over = ref.off(got[t, h], o[at], bound[at], dtype)
        assert not over.any(), (t, h, got[t, h][over][:4], o[at][over][:4], bound[at][over][:4])
        assert abs(got_lse[t, h] - lse[at]) <= lse_bound[at], (t, h, got_lse[t, h], lse[at], lse_bound[at])


def cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("power", [100, 115, -60])
@pytest.mark.parametrize("T,Hq,kernel", [(800, 64, "rows"), (5, 8, "few")])
@pytest.mark.parametrize("D", [64, 128])
def test_values_of_any_size(dev, D, T, Hq, kernel, power):
    """bf16 values by a power of two: the outputs by the same power, not infinities."""
    assert cut(T, 1, Hq, 8, D, T, 900, cus=cus())["kernel"] == kernel
    host = ref.Cache(15, 8, 64, D, 3)
    host.vs *= np.float32(2.0 ** power)
    table = np.random.default_rng(4).permutation(15)[None].astype(np.int32)
    q = torch.randn((T, Hq, D), generator=torch.Generator().manual_seed(5)).bfloat16()
    got = run(dev, q, host, table, [900], [0, T], max_q=T, max_kv=900)
    rows = [(t, h) for t in sorted({0, 1, T // 2, T - 1}) for h in (0, Hq // 2, Hq - 1)]
    close(*got, attention_rows(q.double().numpy(), "bfloat16", host, table, [900], [0, T], rows), "bfloat16", rows)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("B,T,Hq,Hkv,kernel,waves", [(1, 800, 64, 8, "rows", 1), (64, 64, 64, 8, "few", 4)])
def test_many_small_weights_beside_a_large_one(dev, dtype, B, T, Hq, Hkv, kernel, waves):
    """One token with 2^25.05 times the weight of every other and a value of zero: the output is the
    others'.  (Four waves share the tokens of few rows; one of them has the large weight.)"""
    kv, D = 8192, 64
    way = cut(T, B, Hq, Hkv, D, T // B, kv, cus=cus())
    assert way["kernel"] == kernel and not way["share"]
    host = ref.Cache(kv // 64, Hkv, 64, D, 7)
    table = np.random.default_rng(8).permutation(kv // 64)[None].repeat(B, 0).astype(np.int32)
    first = (table[0, 0], slice(None), 0)                    # token 0 of all heads
    host.kc[:], host.ks[:], host.vs[:] = 1, 0, 1
    host.ks[first] = 25.05 * np.log(2.0) / D
    host.vc[:] = 7
    host.vc[first] = 0
    q = torch.ones((T, Hq, D)).to(getattr(torch, dtype))
    lens, cu = [kv] * B, np.arange(B + 1) * (T // B)
    got = run(dev, q, host, table, lens, cu, max_q=T // B, max_kv=kv, scale=1.0)
    rows = [(0, 0), (T // 2, Hq // 2), (T - 1, Hq - 1)]
    want = attention_rows(q.double().numpy(), dtype, host, table, lens, cu, rows, scale=1.0, run=kv // waves)
    assert (want[2] < want[0] / waves).all()                 # (what they lose without the others' weights)
    close(*got, want, dtype, rows)
