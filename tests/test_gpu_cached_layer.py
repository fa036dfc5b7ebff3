"""The attention half of a layer together, as a server uses it: a prompt in parts, then decoding token
by token, eagerly and in a captured step, against the parts' definitions."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import attention_ref as ref  # noqa: E402
from w4a4_group_quantized_amd import apex4  # noqa: E402
from w4a4_group_quantized_amd.attention import BatchPlan, CachedLayerW4A4, KVCache4, rope_frequencies  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    apex4.lib()
    return torch.device("cuda:0")


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_append_then_attend(dev, dtype):
    """Three sequences grow by several tokens a step; every step's output is attention in 64 bits over
    the cache that the definitions say."""
    H, K, D, page = 8, 2, 64, 16
    rng = np.random.default_rng(0)
    cache = KVCache4(40, K, D, page, dev)
    host = ref.Cache.of(*(t.cpu().numpy() for t in cache.tensors))
    table = rng.permutation(40)[:36].reshape(3, 12).astype(np.int32)
    freqs, scale = rope_frequencies(D, scaling="yarn", factor=4.0, original=64, high=32.0, device=dev)
    lens = np.zeros(3, np.int32)
    for step, news in enumerate([(70, 3, 40), (1, 1, 1), (1, 1, 1), (5, 0, 1), (30, 20, 1)]):
        lens = lens + np.array(news, np.int32)
        T = sum(news) + 2                                  # two rows of padding
        cu = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
        plan = BatchPlan(i32(table, dev), i32(lens, dev), i32(cu, dev), page=page, tokens=T, max_q=max(news),
                         max_kv=int(max(lens)))
        g = torch.Generator().manual_seed(step)
        rows = torch.randn((T, H + 2 * K, D), generator=g).to(getattr(torch, dtype))
        on = rows.to(dev)
        q = cache.append(on[:, H:H + K], on[:, H + K:], plan, freqs, on[:, :H], rope_scale=scale)
        out = torch.full_like(q, 3.0)
        cache.attend(q, plan, out=out)
        turned = ref.rope(rows[:, H:H + K].double().numpy(), plan.positions.cpu().numpy(), freqs.cpu().numpy(), False, scale)
        host.put(plan.slots.cpu().numpy(), turned.astype(np.float32), rows[:, H + K:].float().numpy())
        for a, b in zip(host.arrays(), cache.tensors):
            assert np.array_equal(a, b.cpu().numpy())
        want, _, bound, _, owned = ref.attention(q.double().cpu().numpy(), dtype, host, table, lens, cu)
        got = out.double().cpu().numpy()
        assert not ref.off(got[owned], want[owned], bound[owned], dtype).any()
        assert (got[~owned] == 3).all() and (~owned).sum() == 2


def layer(dev, seed=0):
    h, i, heads, kv, D = 256, 384, 4, 2, 64
    g = torch.Generator().manual_seed(seed)
    shapes = {"qkv": ((heads + 2 * kv) * D, h), "o": (h, heads * D), "gate_up": (2 * i, h), "down": (h, i)}
    w = {n: (0.05 * torch.randn(s, generator=g)).half().to(dev) for n, s in shapes.items()}
    return CachedLayerW4A4(w, heads, kv, D, rope_frequencies(D, device=dev)[0])


def test_prompt_in_parts_is_the_prompt(dev):
    """A prompt at once, in two parts, and token by token: the cache to the bit, the rows within what
    the calls' different shares of the tokens may change (a rounding of the attention's output can
    move one 4-bit code of O's input: a seventh of a group's largest, times the weights)."""
    m = layer(dev)
    x = torch.randn((48, 256), generator=torch.Generator().manual_seed(1)).half().to(dev)
    table = i32([[2, 0, 3]], dev)
    outs, caches = [], []
    for parts in ([48], [31, 17], [1] * 48):
        cache, at, rows = KVCache4(4, 2, 64, 16, dev), 0, []
        for n in parts:
            plan = BatchPlan(table, i32([at + n], dev), i32([0, n], dev), page=16, tokens=n, max_q=n, max_kv=48)
            rows.append(m(x[at:at + n], cache, plan))
            at += n
        outs.append(torch.cat(rows))
        caches.append(cache)
    for c in caches[1:]:
        for a, b in zip(caches[0].tensors, c.tensors):
            assert torch.equal(a, b)
    for y in outs[1:]:
        assert torch.isfinite(y).all()
        # most rows are the same to the bit or a step; none is another row
        assert (y.float() - outs[0].float()).abs().median() <= 2 ** -9 * outs[0].float().abs().max()


def test_captured_decode_step(dev):
    """One decoding step of a padded batch, captured and replayed while the sequences grow."""
    m = layer(dev, 3)
    B, page = 5, 16
    table = i32([[0, 1], [2, 3], [4, 5], [6, 7], [-1, -1]], dev)      # the last place of the batch is empty
    lens = i32([3, 15, 1, 9, 0], dev)
    eager, graphed = KVCache4(8, 2, 64, page, dev), KVCache4(8, 2, 64, page, dev)
    x = torch.randn((B, 256), generator=torch.Generator().manual_seed(5)).half().to(dev)

    def step(cache):
        plan = BatchPlan(table, lens, page=page, max_kv=2 * page)
        return m(x, cache, plan)

    start = lens.clone()
    step(graphed)                                          # (warm: workspaces, library)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = step(graphed)
    for t in graphed.tensors:
        t.zero_()
    for n in range(4):
        x.copy_(torch.randn((B, 256), generator=torch.Generator().manual_seed(n)).half())
        lens.copy_(start + n * (start > 0))
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        want = step(eager)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        for a, b in zip(eager.tensors, graphed.tensors):
            assert torch.equal(a, b)


def test_refusals(dev):
    m = layer(dev)
    w = {"qkv": torch.zeros((256, 256), dtype=torch.float16, device=dev)}
    for name in ("o", "gate_up", "down"):
        w[name] = torch.zeros((256, 256), dtype=torch.float16, device=dev)
    with pytest.raises(ValueError):
        CachedLayerW4A4(w, 4, 2, 64, m.inv_freq)
    plan = BatchPlan(i32([[0]], dev), i32([1], dev), page=32)
    with pytest.raises(ValueError):
        m(torch.zeros((1, 256), dtype=torch.float16, device=dev), KVCache4(2, 2, 64, 16, dev), plan)
