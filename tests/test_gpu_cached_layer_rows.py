"""CachedLayerW4A4 row by row: against its parts' definitions put together, and a prompt in parts against the prompt."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import attention_ref as ref  # noqa: E402
from w4a4_group_quantized_amd import apex4  # noqa: E402
from w4a4_group_quantized_amd.attention import BatchPlan, CachedLayerW4A4, KVCache4, rope_frequencies  # noqa: E402

pytestmark = pytest.mark.gpu
HEADS, KV, D, HIDDEN, INTER, GROUP = 4, 2, 64, 256, 384, 128


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    apex4.lib()
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def layer(dev):
    g = torch.Generator().manual_seed(0)
    shapes = {"qkv": ((HEADS + 2 * KV) * D, HIDDEN), "o": (HIDDEN, HEADS * D), "gate_up": (2 * INTER, HIDDEN),
              "down": (HIDDEN, INTER)}
    w = {n: (0.05 * torch.randn(s, generator=g)).half().to(dev) for n, s in shapes.items()}
    return CachedLayerW4A4(w, HEADS, KV, D, rope_frequencies(D, device=dev)[0], GROUP)


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def composed(m, x, host, plan, table, lens, cu):
    """The layer's forward with its own linears (tested for themselves) and the rotation, cache and
    attention of attention_ref in between, rounded where the layer's are.  (outputs, attention's
    output, its bound)"""
    rows = m.qkv(x).view(len(x), HEADS + 2 * KV, D)
    parts = rows.double().cpu().numpy()
    freqs, pos = m.inv_freq.cpu().numpy(), plan.positions.cpu().numpy()
    turned = ref.rope(parts[:, :HEADS + KV], pos, freqs).astype(np.float32)
    q = torch.from_numpy(turned[:, :HEADS]).half()
    host.put(plan.slots.cpu().numpy(), turned[:, HEADS:], parts[:, HEADS + KV:].astype(np.float32))
    o, _, bound, _, owned = ref.attention(q.double().numpy(), "float16", host, table, lens, cu)
    return q, o, bound, owned


def finish(m, x, o):
    x = x + m.o(o.reshape(len(x), -1))
    gu = m.gate_up(x)
    return x + m.down(torch.nn.functional.silu(gu[:, :INTER]) * gu[:, INTER:])


def test_layer_is_its_parts(dev, layer, monkeypatch):
    """Three uneven sequences and padding: the attention that the layer runs is the definitions' within
    their bound in every row, its cache theirs to the bit, and its output the one of its other parts
    on that attention, to the bit."""
    seen = []
    attend = KVCache4.attend

    def spy(self, q, plan, **args):
        seen.append((q.clone(), attend(self, q, plan, **args)))
        return seen[-1][1]

    monkeypatch.setattr(KVCache4, "attend", spy)
    cache = KVCache4(12, KV, D, 16, dev)
    host = ref.Cache.of(*(t.cpu().numpy() for t in cache.tensors))
    table = np.random.default_rng(3).permutation(12).reshape(3, 4).astype(np.int32)
    lens = np.zeros(3, np.int32)
    for step, news in enumerate([(20, 1, 33), (1, 1, 1), (3, 0, 17)]):
        lens = lens + np.array(news, np.int32)
        cu = np.concatenate(([2], 2 + np.cumsum(news))).astype(np.int32)
        T = int(cu[-1]) + 3
        plan = BatchPlan(i32(table, dev), i32(lens, dev), i32(cu, dev), page=16, tokens=T, max_q=max(news), max_kv=64)
        x = torch.randn((T, HIDDEN), generator=torch.Generator().manual_seed(step)).half().to(dev)
        y = layer(x, cache, plan)
        q, o, bound, owned = composed(layer, x, host, plan, table, lens, cu)
        (got_q, got_o), = seen
        seen.clear()
        for a, b in zip(host.arrays(), cache.tensors):
            assert np.array_equal(a, b.cpu().numpy())
        assert torch.equal(got_q.cpu(), q)
        assert not ref.off(got_o.double().cpu().numpy(), o, bound, "float16")[owned].any()
        assert (got_o[torch.from_numpy(~owned).to(dev)] == 0).all()
        assert torch.equal(y, finish(layer, x, got_o))


def test_every_row_of_a_prompt_in_parts(dev, layer):
    """A prompt at once, in two parts, and token by token.  The parts' attention differs by roundings,
    which move one 4-bit code in some hundreds to its neighbour.  One in every group of 128 is allowed: it is
    a seventh of the group's largest, 0.4 of its root mean square, so sqrt(1 / 128) 0.4 = 0.035 of the
    input's norm; O, gate and up, and down bring three of those, 0.1 of the row.  No row is another one."""
    x = torch.randn((48, HIDDEN), generator=torch.Generator().manual_seed(1)).half().to(dev)
    table, outs = i32([[2, 0, 3]], dev), []
    for parts in ([48], [31, 17], [1] * 48):
        cache, at, rows = KVCache4(4, KV, D, 16, dev), 0, []
        for n in parts:
            plan = BatchPlan(table, i32([at + n], dev), i32([0, n], dev), page=16, tokens=n, max_q=n, max_kv=48)
            rows.append(layer(x[at:at + n], cache, plan))
            at += n
        outs.append(torch.cat(rows).double())
    size = outs[0].norm(dim=-1)
    apart = torch.cdist(outs[0], outs[0]) + torch.diag(torch.full((48,), float("inf"), device=dev, dtype=torch.float64))
    for y in outs[1:]:
        off = (y - outs[0]).norm(dim=-1)
        assert (off <= 0.1 * size).all() and (off < 0.1 * apart.amin(-1)).all(), (off / size).max()
