"""apex4_kv4_append and apex4_kv4_read against the cache's definition on the host: codes and scales
to the bit."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import attention_ref as ref  # noqa: E402
from w4a4_group_quantized_amd import apex4  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    apex4.lib()
    return torch.device("cuda:0")


def gpu(dev, cache):
    return tuple(torch.from_numpy(a).to(dev) for a in cache.arrays())


def same(cache, tensors):
    got = [t.cpu().numpy() for t in tensors]
    for a, b, name in zip(cache.arrays(), got, ("k_codes", "k_scales", "v_codes", "v_scales")):
        assert np.array_equal(a, b, equal_nan=a.dtype.kind == "f"), name


def numbers(T, H, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H, D), generator=g)
    x[:, :, 7] *= 20                                   # a channel that stands out
    return x.to(getattr(torch, dtype))


def places(rng, n, pages, page, dropped=0):
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    slots[n - dropped:] = -1
    return slots


SHAPES = [  # T, Hq, Hkv, D, page, R, interleaved
    (1, 32, 32, 128, 16, 128, False), (1, 1, 1, 64, 16, 64, True), (5, 8, 2, 128, 64, 64, True),
    (17, 6, 3, 256, 32, 256, False), (61, 64, 8, 128, 64, 128, False), (130, 4, 4, 64, 1024, 16, False),
    (300, 5, 1, 128, 16, 96, True), (600, 2, 2, 64, 128, 48, False)]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("T,Hq,Hkv,D,page,R,interleaved", SHAPES)
def test_append_and_read(dev, dtype, T, Hq, Hkv, D, page, R, interleaved):
    rng = np.random.default_rng(T + D)
    pages = -(-T // page) + 3
    host = ref.Cache(pages, Hkv, page, D, seed=T)
    cache = gpu(dev, host)
    rows = numbers(T, Hq + 2 * Hkv, D, dtype, T)
    slots = places(rng, T, pages, page, T // 5)
    positions = rng.integers(0, 2 ** 17, T)
    freqs = ref.frequencies(R)
    turn = dict(positions=torch.from_numpy(positions).to(dev), inv_freq=torch.from_numpy(freqs).to(dev),
                interleaved=interleaved, rope_scale=1.1)
    on = rows.to(dev)
    at = torch.from_numpy(slots).to(dev)
    q = apex4.kv4_append(cache, on[:, Hq:Hq + Hkv], on[:, Hq + Hkv:], at, q=on[:, :Hq], **turn)
    turned = ref.rope(rows[:, :Hq + Hkv].double().numpy(), positions, freqs, interleaved, 1.1)
    want = turned[:, :Hq]
    bound = ref.rounding(want, dtype) + ref.rounding(want, "float32") + np.abs(want).max() * 2.0 ** -46
    assert (np.abs(q.double().cpu().numpy() - want) <= bound).all()
    host.put(slots, turned[:, Hq:].astype(np.float32), rows[:, Hq + Hkv:].float().numpy())
    same(host, cache)
    # in any order, some twice, some outside
    seek = np.concatenate((slots[::-1], [-1, pages * page, 2 ** 62, -2 ** 62], rng.integers(0, pages * page, 33)))
    for out in ("float32", "float16", "bfloat16"):
        got = apex4.kv4_read(cache, torch.from_numpy(seek).to(dev), getattr(torch, out))
        for a, b in zip(got, host.values(seek)):
            if out == "float32":
                assert torch.equal(a.cpu(), torch.from_numpy(b).float())
            else:
                # code times scale, rounded to the type at once or by way of fp32
                bound = ref.rounding(b, out) + ref.rounding(b, "float32")
                assert (np.abs(a.double().cpu().numpy() - b) <= bound).all(), out
    # one token at a time gives the same bytes
    again = gpu(dev, ref.Cache(pages, Hkv, page, D, seed=T))
    for t in range(min(T, 40)):
        one = dict(turn, positions=turn["positions"][t:t + 1])
        r = apex4.kv4_append(again, on[t:t + 1, Hq:Hq + Hkv], on[t:t + 1, Hq + Hkv:], at[t:t + 1], q=on[t:t + 1, :Hq],
                             **one)
        assert torch.equal(r, q[t:t + 1])
    if T <= 40:
        same(host, again)


def test_append_without_rotation_or_queries(dev):
    T, H, D, page = 37, 3, 128, 32
    host = ref.Cache(3, H, page, D)
    cache = gpu(dev, host)
    k, v = (numbers(T, H, D, "float16", i).to(dev) for i in (1, 2))
    slots = places(np.random.default_rng(0), T, 3, page)
    assert apex4.kv4_append(cache, k, v, torch.from_numpy(slots).to(dev)) is None
    host.put(slots, k.float().cpu().numpy(), v.float().cpu().numpy())
    same(host, cache)
    pos = torch.arange(T, device=dev)
    freqs = ref.frequencies(D)
    assert apex4.kv4_append(cache, k, v, torch.from_numpy(slots).to(dev), positions=pos,
                            inv_freq=torch.from_numpy(freqs).to(dev)) is None
    turned = ref.rope(k.double().cpu().numpy(), np.arange(T), freqs)
    host.put(slots, turned.astype(np.float32), v.float().cpu().numpy())
    same(host, cache)


def test_queries_in_place(dev):
    T, D = 6, 64
    q, k = numbers(T, 4, D, "float16", 1).to(dev), numbers(T, 1, D, "float16", 2).to(dev)
    cache = apex4.kv4_cache(2, 1, D, 16, dev)
    args = dict(positions=torch.arange(T, device=dev), inv_freq=torch.from_numpy(ref.frequencies(D)).to(dev))
    slots = torch.arange(T, device=dev)
    want = apex4.kv4_append(cache, k, k, slots, q=q, **args)
    assert apex4.kv4_append(cache, k, k, slots, q=q, q_out=q, **args) is q
    assert torch.equal(q, want)


def test_numbers_at_the_ends(dev):
    """Zeros, ties, the largest and smallest numbers, and numbers that are not finite: their head only."""
    D, page = 64, 16
    k = torch.randn((14, 2, D), generator=torch.Generator().manual_seed(5)).bfloat16()
    k[0] = 0
    k[1, 0, 0] = float("nan")
    k[2, 0, 63] = float("inf")
    k[3, 1, 31] = float("-inf")
    k[4] = torch.finfo(torch.bfloat16).max
    k[5] = 0
    k[5, :, ::3] = 2.0 ** -133                                     # the smallest: its seventh rounds to nothing
    k[6] = 0
    k[6, :, 0], k[6, :, 1:8] = 7, torch.tensor([0.5, 1.5, 2.5, -0.5, -1.5, -2.5, -7.0])
    k[7] = -0.0
    k[8] *= 2.0 ** 100
    k[9] *= 2.0 ** -110
    k[10] = 0
    k[10, :, :6] = torch.tensor([10, -10, 9, -9, 4, 3]) * 2.0 ** -133   # scale of 1 smallest step (of fp32: 2^-149 * 2^16)
    v = k.flip(0).contiguous()
    host = ref.Cache(1, 2, page, D)
    cache = gpu(dev, host)
    slots = np.arange(14)[::-1].copy()
    apex4.kv4_append(cache, k.to(dev), v.to(dev), torch.from_numpy(slots).to(dev))
    host.put(slots, k.float().numpy(), v.float().numpy())
    same(host, cache)


def test_cache_beyond_32_bits(dev):
    """Places behind 2^32 bytes of codes: pages of 8 heads of 128 numbers, 64 tokens each, are 32 KB."""
    pages, H, D, page = 140000, 8, 128, 64                         # 4.6 GB of codes each for keys and values
    if torch.cuda.mem_get_info()[0] < 14 << 30:
        pytest.skip("not enough memory")
    cache = apex4.kv4_cache(pages, H, D, page, dev)
    slots = torch.tensor([pages * page - 1, 131072 * page + 5, 131071 * page + 63, 0, 17], device=dev)
    k, v = numbers(5, H, D, "float16", 1).to(dev), numbers(5, H, D, "float16", 2).to(dev)
    apex4.kv4_append(cache, k, v, slots)
    got = apex4.kv4_read(cache, slots, torch.float32)
    for x, y in zip((k, v), got):
        c, s = ref.codes(x.float().cpu().numpy())
        assert torch.equal(y.cpu(), torch.from_numpy((c * s.astype(np.float64)[..., None])).float())
    # nothing else was written
    assert int((cache[1] != 0).sum()) == 5 * H and int((cache[3] != 0).sum()) == 5 * H
    assert not cache[0].view(-1)[1 << 20:(1 << 20) + (1 << 24)].any()
    q = numbers(1, H, D, "float16", 3).to(dev)
    table = torch.tensor([[pages - 1, 131071]], dtype=torch.int32, device=dev)
    o = apex4.kv4_attention(q, cache, table, torch.tensor([128], dtype=torch.int32, device=dev))
    small = tuple(t[[pages - 1, 131071]].contiguous() for t in cache)
    table = torch.tensor([[0, 1]], dtype=torch.int32, device=dev)
    assert torch.equal(o, apex4.kv4_attention(q, small, table, torch.tensor([128], dtype=torch.int32, device=dev)))


def test_refusals(dev):
    cache = apex4.kv4_cache(4, 2, 64, 16, dev)
    k = torch.zeros((3, 2, 64), dtype=torch.float16, device=dev)
    slots = torch.arange(3, device=dev)
    pos, freq = torch.arange(3, device=dev), torch.zeros(32, dtype=torch.float64, device=dev)
    with pytest.raises(ValueError):
        apex4.kv4_cache(4, 2, 100, 16, dev)
    for bad in (dict(k=k.float()), dict(k=k[:, :1]), dict(k=k.cpu()), dict(v=k.bfloat16()), dict(v=k[:2]),
                dict(slots=slots.int()), dict(slots=slots[:2]), dict(positions=pos), dict(inv_freq=freq), dict(q=k),
                dict(q_out=k), dict(q=k.bfloat16(), positions=pos, inv_freq=freq),
                dict(q=k[:2], positions=pos, inv_freq=freq), dict(cache=cache[:2] + cache[:2]),
                dict(cache=(cache[0], cache[1][:2], cache[2], cache[3]))):
        with pytest.raises(ValueError):
            apex4.kv4_append(**{**dict(cache=cache, k=k, v=k, slots=slots), **bad})
    with pytest.raises(ValueError):
        apex4.kv4_read(cache, slots.int())
    with pytest.raises(ValueError):
        apex4.kv4_read(cache, slots, torch.float64)
    assert apex4.kv4_read(cache, slots[:0])[0].shape == (0, 2, 64)
    assert apex4.kv4_append(cache, k[:0], k[:0], slots[:0]) is None


@pytest.mark.parametrize("dtype,D,T", [("float16", 128, 40001), ("bfloat16", 64, 70003), ("float32", 64, 40001),
                                       ("float32", 128, 20001), ("bfloat16", 256, 20001)])
def test_reads_beyond_the_caches(dev, dtype, D, T):
    """More than 128 MB of values: the bits of the same tokens read in parts, and nothing beside them."""
    dtype = getattr(torch, dtype)
    cache = apex4.kv4_cache(33, 8, D, 64)
    g = torch.Generator(device=dev).manual_seed(D)
    for c in cache:
        if c.dtype == torch.uint8:
            c.random_(0, 256, generator=g)
        else:
            c.uniform_(0.01, 1.0, generator=g)
    slots = torch.randint(-5, 33 * 64 + 5, (T,), device=dev, generator=g)
    room = [torch.full((T + 2, 8, D), 7.0, dtype=dtype, device=dev) for _ in range(2)]
    apex4.kv4_read(cache, slots, dtype, out=tuple(x[1:-1] for x in room))
    parts = [apex4.kv4_read(cache, s, dtype) for s in slots.split(5000)]
    for x, y in zip(room, zip(*parts)):
        assert torch.equal(x[1:-1], torch.cat(y)) and (x[[0, -1]] == 7).all()
