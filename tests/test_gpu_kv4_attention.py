"""apex4_kv4_attention against attention in 64 bits over the values that the cache's codes stand for."""
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


def make(news, olds, heads, D, page, seed=0, extra=2):
    """A filled cache on the host, a shuffled table (unused entries are not pages) and cu_q."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in olds]
    pages = sum(need) + extra
    host = ref.Cache(pages, heads, page, D, seed + 1)
    order = rng.permutation(pages)
    table = np.full((len(olds), max(1, max(need))), -7, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return host, table, np.concatenate(([0], np.cumsum(news))).astype(np.int32)


def queries(T, H, D, dtype, seed=0, size=1.3):
    g = torch.Generator().manual_seed(seed)
    return (size * torch.randn((T, H, D), generator=g)).to(getattr(torch, dtype))


def run(dev, q, host, table, olds, cu, **args):
    to = lambda a, t=None: torch.as_tensor(np.asarray(a), dtype=t).to(dev)  # noqa: E731
    cache = tuple(to(a) for a in host.arrays())
    T, H, D = q.shape
    out = torch.full((T + 2, H, D), 7.0, dtype=q.dtype, device=dev)
    lse = torch.full((T + 2, H), 7.0, device=dev)
    rest = (cache, to(table, torch.int32), to(olds, torch.int32), None if cu is None else to(cu, torch.int32))
    apex4.kv4_attention(q.to(dev), *rest, want_lse=True, out=out[1:-1], lse=lse[1:-1], **args)
    torch.cuda.synchronize()
    assert (out[[0, -1]] == 7).all() and (lse[[0, -1]] == 7).all()          # rows beside the call's
    return out[1:-1].double().cpu().numpy(), lse[1:-1].double().cpu().numpy()


def check(dev, dtype, q, host, table, olds, cu, max_q=None, max_kv=None, **args):
    got, got_lse = run(dev, q, host, table, olds, cu, max_q=max_q, max_kv=max_kv, **args)
    want, lse, bound, lse_bound, owned = ref.attention(q.double().numpy(), dtype, host, table, olds, cu, **args)
    assert (got[~owned] == 7).all() and (got_lse[~owned] == 7).all()
    got, want, bound, got_lse, lse, lse_bound = (a[owned] for a in (got, want, bound, got_lse, lse, lse_bound))
    nan = np.isnan(want).any(-1)
    assert np.isnan(got[nan]).any(-1).all()
    over = ref.off(got, want, bound, dtype) & ~nan[..., None]
    assert not over.any(), (np.argwhere(over)[:4], np.abs(got - want)[over].max(), bound[over][:4])
    none = np.isneginf(lse)
    assert (got[none] == 0).all() and np.isneginf(got_lse[none]).all()
    live = ~none & ~nan & np.isfinite(lse)
    assert (np.abs(got_lse[live] - lse[live]) <= lse_bound[live]).all()


CASES = [  # new tokens, cached tokens, query heads, key heads, D, page
    ([1], [1], 1, 1, 64, 16), ([1], [16], 4, 4, 128, 16), ([1], [517], 8, 8, 128, 16), ([1], [63], 8, 1, 256, 64),
    ([1, 1, 1], [65, 1, 300], 16, 2, 128, 32), ([1] * 9, [5, 0, 64, 128, 129, 200, 1, 33, 0], 10, 2, 64, 16),
    ([1], [5000], 8, 2, 128, 128), ([1, 1], [2300, 7], 64, 1, 128, 64), ([1], [1111], 7, 1, 64, 1024),
    ([5], [5], 4, 2, 128, 16), ([16], [16], 2, 2, 64, 16), ([3, 1, 40], [3, 70, 129], 6, 3, 128, 32),
    ([100], [100], 3, 1, 256, 64), ([33, 1, 65], [400, 90, 65], 16, 4, 64, 32), ([130], [700], 8, 8, 128, 64),
    ([257], [300], 5, 1, 128, 128), ([2, 70], [2048, 71], 8, 1, 128, 256), ([300, 20], [300, 900], 2, 1, 256, 16),
    ([17], [1500], 1, 1, 128, 16), ([600], [600], 2, 2, 64, 64)]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("news,olds,Hq,Hkv,D,page", CASES)
def test_against_64_bits(dev, dtype, news, olds, Hq, Hkv, D, page):
    host, table, cu = make(news, olds, Hkv, D, page, sum(olds))
    q = queries(sum(news), Hq, D, dtype, len(olds) + Hq)
    one = max(news) == 1
    check(dev, dtype, q, host, table, olds, None if one else cu, max_q=max(news), max_kv=max(1, max(olds)))
    if one:
        check(dev, dtype, q, host, table, olds, cu)


@pytest.mark.parametrize("causal,window", [(True, 1), (True, 17), (True, 64), (True, 1000), (False, 0)])
@pytest.mark.parametrize("news,olds,Hq,Hkv,D,page", [
    ([1, 1, 1], [65, 1, 300], 8, 2, 128, 32), ([1], [2100], 4, 1, 64, 64), ([40, 3], [129, 3], 6, 3, 128, 32),
    ([200, 1], [1300, 900], 8, 2, 64, 16), ([150], [150], 2, 1, 256, 64)])
def test_masks(dev, causal, window, news, olds, Hq, Hkv, D, page):
    host, table, cu = make(news, olds, Hkv, D, page, sum(olds) + window)
    q = queries(sum(news), Hq, D, "float16", window)
    check(dev, "float16", q, host, table, olds, cu, max_q=max(news), causal=causal, window=window)


def test_queries_ahead_of_the_cache_see_nothing(dev):
    """More new queries than cached tokens: the first ones stand before the first token."""
    host, table, cu = make([9, 5, 4], [4, 0, 70], 2, 64, 16, 1)
    q = queries(18, 4, 64, "float16")
    check(dev, "float16", q, host, table, [4, 0, 70], cu)
    check(dev, "float16", q, host, table, [4, -3, 70], cu, window=2)
    check(dev, "float16", q, host, table, [4, 0, 70], cu, causal=False)


def test_the_widest_window_is_none(dev):
    """Also for queries before the first token, whose position less the window passes 32 bits."""
    host, table, cu = make([9, 40, 300], [4, 11, 290], 2, 64, 16, 18)
    q = queries(349, 4, 64, "float16")
    check(dev, "float16", q, host, table, [4, 11, 290], cu, window=2 ** 31 - 1)
    check(dev, "float16", q[:9], host, table[:1], [4], cu[:2], window=2 ** 31 - 1)


@pytest.mark.parametrize("news", [[1, 1, 1], [30, 1, 90]])
def test_pages_that_are_none(dev, news):
    """Numbers outside the cache are pages that hold nothing: not seen, not read."""
    olds = [200, 64, 500]
    host, table, cu = make(news, olds, 2, 128, 16, 3)
    table[0, 3] = -1
    table[0, 5:9] = 2 ** 31 - 1
    table[1, :] = len(host.kc)
    table[2, 0:20] = -2 ** 31
    table[2, 25] = len(host.kc) - 1 - table[2, 25] if table[2, 25] < 0 else table[2, 26]     # a page twice
    check(dev, "float16", queries(sum(news), 4, 128, "float16"), host, table, olds, cu, max_q=max(news))


@pytest.mark.parametrize("news", [[1, 1], [20, 33], [140, 33]])
def test_what_is_behind_a_sequence_stays_unseen(dev, news):
    """NaN scales in the places that no token has, in whole pages and inside the last one."""
    olds = [150, 333]
    host, table, cu = make(news, olds, 2, 64, 64, 4)
    used = np.zeros(host.ks.shape[0::2], bool)
    for b, n in enumerate(olds):
        for j in range(n):
            used[table[b, j // 64], j % 64] = True
    for s in (host.ks, host.vs):
        s.transpose(0, 2, 1)[~used] = np.nan
    check(dev, "bfloat16", queries(sum(news), 4, 64, "bfloat16"), host, table, olds, cu, max_q=max(news))


@pytest.mark.parametrize("news", [[1, 1], [40, 90], [200, 90]])
def test_what_is_not_finite_shows_in_its_rows_only(dev, news):
    olds = [300, 222]
    host, table, cu = make(news, olds, 2, 128, 16, 5)
    host.ks[table[0, 295 // 16], 1, 295 % 16] = np.nan            # seen by the last rows of sequence 0, head 1
    host.vs[table[1, 3], 0, 5] = np.nan                           # seen by (nearly) all rows of sequence 1, head 0
    q = queries(sum(news), 4, 128, "float16")
    q[0, 0, 17] = float("nan")
    q[-1, 2, 3] = float("inf")
    clean = q.clone()
    clean[0, 0, 17] = clean[-1, 2, 3] = 0
    got, _ = run(dev, q, host, table, olds, cu, max_q=max(news))
    bad = np.isnan(got).any(-1)
    assert bad[0, 0] and bad[-1, 2]
    check(dev, "float16", clean, host, table, olds, cu, max_q=max(news))
    other, _ = run(dev, clean, host, table, olds, cu, max_q=max(news))
    mine = np.zeros(bad.shape, bool)
    mine[0, 0] = mine[-1, 2] = True
    assert np.array_equal(got[~mine], other[~mine], equal_nan=True)      # the other rows keep their bits


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("news", [[1], [50], [260]])
def test_sizes_far_apart(dev, dtype, news):
    """Values' scales over 40 powers of two and zeros among them, keys of scale zero, rows of
    queries from tiny to huge in one call (bf16), zeros."""
    olds = [700]
    host, table, cu = make(news, olds, 1, 128, 64, 6)
    rng = np.random.default_rng(7)
    host.vs *= np.exp2(rng.integers(-20, 20, host.vs.shape)).astype(np.float32)
    host.vs[rng.random(host.vs.shape) < 0.2] = 0
    host.ks[rng.random(host.ks.shape) < 0.1] = 0
    q = queries(news[0], 4, 128, dtype)
    q[:, 1] = 0
    if dtype == "bfloat16":
        q[:, 2] *= 2.0 ** 30
        host.ks *= 0.25
    q[:, 3] *= 2.0 ** -9
    check(dev, dtype, q, host, table, olds, cu, max_q=news[0])


@pytest.mark.parametrize("news", [[1], [70]])
def test_all_values_zero_or_one_token_above_all(dev, news):
    host, table, cu = make(news, [400], 2, 64, 16, 8)
    host.vs[:, 0] = 0
    host.ks[table[0, 10], 1, 3] = 300.0                           # scores of hundreds
    check(dev, "float16", queries(news[0], 4, 64, "float16"), host, table, [400], cu, max_q=news[0])


@pytest.mark.parametrize("tops", [40.0, -40.0])
@pytest.mark.parametrize("news", [[1], [64]])
def test_scores_that_rise_or_fall_along_the_cache(dev, tops, news):
    """The running maximum moves with every tile, or never after the first."""
    host, table, cu = make(news, [1500], 1, 64, 64, 9)
    j = np.arange(1500)
    host.kc[:, :, :, :] = 1
    rise = (np.linspace(0, tops, 1500) / 64).astype(np.float32)
    host.ks[table[0, j // 64], 0, j % 64] = rise
    q = torch.full((news[0], 2, 64), 1.0).half()
    check(dev, "float16", q, host, table, [1500], cu, max_q=news[0], scale=1.0)


@pytest.mark.parametrize("max_q,max_kv", [(1, 1), (1, 100000), (3, 64), (4096, 16), (4096, 4096)])
def test_expected_sizes_only_split_the_work(dev, max_q, max_kv):
    news, olds = [70, 1, 200], [900, 2500, 200]
    host, table, cu = make(news, olds, 2, 128, 64, 10)
    q = queries(sum(news), 8, 128, "float16")
    check(dev, "float16", q, host, table, olds, cu, max_q=max_q, max_kv=max_kv)


def test_rows_behind_the_last_sequence_and_parts_of_a_projection(dev):
    """A padded batch: queries that no sequence owns keep their output; q is a slice of a wider row."""
    news, olds = [3, 40], [10, 200]
    host, table, cu = make(news, olds, 2, 64, 32, 11)
    rows = queries(60, 8, 64, "bfloat16").to(dev)
    to = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(dev)  # noqa: E731
    cache = tuple(torch.from_numpy(a).to(dev) for a in host.arrays())
    out = torch.full((60, 4, 64), 7.0, dtype=torch.bfloat16, device=dev)
    apex4.kv4_attention(rows[:, 2:6], cache, to(table), to(olds), to(cu), out=out, max_q=40)
    assert (out[43:] == 7).all()
    want = apex4.kv4_attention(rows[:43, 2:6].contiguous(), cache, to(table), to(olds), to(cu), max_q=40)
    assert torch.equal(out[:43], want)
    # entries of cu_q beyond the call's rows end with them
    wide = to([0, 3, 2 ** 31 - 1])
    apex4.kv4_attention(rows[:, 2:6], cache, to(table), to(olds), wide, out=out, max_q=40)
    assert torch.isfinite(out.float()).all()


def uneven(kind):
    """(new tokens, cached tokens, query heads, key heads, window): prompts among sequences of few tokens."""
    rng = np.random.default_rng(len(kind))
    news = rng.integers(0, 3, 70)
    olds = news + rng.integers(0, 200, 70)
    if kind.startswith("many rows"):
        news[[3, 64]] = 900, 811
        olds[[3, 64]] = 900, 1000
        return news, olds, 16, 4, 90 * kind.endswith("window")
    if kind == "many sequences":
        news = (np.arange(4500) % 3 == 1).astype(int)
        olds = news + np.arange(4500) % 2
        news[[0, 4095, 4499]] = 300, 129, 140
        olds[[0, 4095, 4499]] = 300, 200, 140
        return news, olds, 1, 1, 0
    news[[0, 69]] = 60, 33
    olds[[0, 69]] = {"few rows": (70, 1200), "shared": (2500, 100), "window": (2500, 2100)}[kind]
    return news, olds, 16, 4, 1100 if kind == "window" else 0


@pytest.mark.parametrize("kind", ["many rows", "many rows, window", "few rows", "shared", "window", "many sequences"])
def test_prompts_among_sequences_of_few_tokens(dev, kind):
    """Row tiles are numbered over all sequences; rows before the first and behind the last have none."""
    news, olds, Hq, Hkv, window = uneven(kind)
    host, table, cu = make(list(news), list(olds), Hkv, 64, 16, 17)
    q = queries(int(cu[-1]) + 50, Hq, 64, "float16", 17)
    check(dev, "float16", q, host, table, olds, cu + 37, max_q=int(max(news)), max_kv=int(max(olds)), window=window)
    if not kind.startswith("many rows"):                         # (a guess too low costs time only)
        check(dev, "float16", q, host, table, olds, cu + 37, max_q=1, max_kv=1, window=window)


def test_same_bits_every_time_and_alone(dev):
    """The same call twice gives the same bits; on another stream too; a sequence's rows do not
    depend on the other queries, or on their pages' contents, in a call of the same lengths."""
    news, olds = [1] * 6, [3000, 10, 640, 64, 63, 1025]
    host, table, _ = make(news, olds, 2, 128, 64, 12)
    q = queries(6, 16, 128, "float16")
    first, _ = run(dev, q, host, table, olds, None, max_kv=3000)
    again, _ = run(dev, q, host, table, olds, None, max_kv=3000)
    assert np.array_equal(first, again)
    other = q.clone()
    other[1:] = 0
    elsewhere = table.copy()
    elsewhere[1:] = table[0]
    alone, _ = run(dev, other, host, elsewhere, olds, None, max_kv=3000)
    assert np.array_equal(first[0], alone[0])
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        on, _ = run(dev, q, host, table, olds, None, max_kv=3000)
    assert np.array_equal(first, on)


@pytest.mark.parametrize("news,olds", [([1, 1, 1], [4000, 5, 700]), ([90, 1], [300, 2000])])
def test_graph(dev, news, olds):
    """Captured once, replayed with other queries, lengths and pages, with eager work between."""
    host, table, cu = make(news, olds, 2, 128, 64, 13)
    T = sum(news)
    to = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(dev)  # noqa: E731
    cache = tuple(torch.from_numpy(a).to(dev) for a in host.arrays())
    q, tab, lens, cu_q = queries(T, 8, 128, "float16").to(dev), to(table), to(olds), to(cu)
    args = dict(max_q=max(news), max_kv=max(olds), want_lse=True)
    apex4.kv4_attention(q, cache, tab, lens, cu_q, **args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = apex4.kv4_attention(q, cache, tab, lens, cu_q, **args)
    for i in range(4):
        q.copy_(queries(T, 8, 128, "float16", i + 20))
        lens.copy_(to([max(n, (o_ * (i + 1)) // 4) for n, o_ in zip(news, olds)]))
        g.replay()
        torch.cuda.synchronize()
        got, got_lse = o.clone(), lse.clone()
        want, want_lse = apex4.kv4_attention(q, cache, tab, lens, cu_q, **args)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(got_lse, want_lse)


def test_refusals(dev):
    cache = apex4.kv4_cache(4, 2, 64, 16, dev)
    q = torch.zeros((2, 4, 64), dtype=torch.float16, device=dev)
    table, lens = torch.zeros((2, 3), dtype=torch.int32, device=dev), torch.ones(2, dtype=torch.int32, device=dev)
    base = dict(q=q, cache=cache, table=table, kv_lens=lens)
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[..., :32]), dict(q=q.transpose(1, 2)), dict(table=table[0]),
                dict(table=table.long()), dict(kv_lens=lens[:1]), dict(kv_lens=lens.long()), dict(cu_q=lens),
                dict(out=q[:1]), dict(out=q.bfloat16()), dict(lse=lens), dict(workspace=lens), dict(max_q=2 ** 31),
                dict(max_kv=-1), dict(window=-1), dict(cache=(cache[0], cache[1], cache[2][:3], cache[3]))):
        with pytest.raises(ValueError):
            apex4.kv4_attention(**{**base, **bad})
    for bad in (dict(q=q[:1]), dict(window=3, causal=False), dict(scale=float("nan")), dict(max_q=0),
                dict(q=torch.zeros((2, 3, 64), dtype=torch.float16, device=dev))):
        with pytest.raises(apex4.Apex4Error):
            apex4.kv4_attention(**{**base, **bad})
    assert apex4.kv4_attention(q[:0], cache, table[:0], lens[:0]).shape == (0, 4, 64)


def test_more_sequences_than_a_workgroup_sorts(dev):
    """300 sequences of one key head: shared out by a sum over all lengths; and 600: whole, unsorted."""
    for B, longest in ((300, 2000), (600, 1700)):
        rng = np.random.default_rng(B)
        olds = [int(x) for x in rng.integers(0, 40, B)]
        olds[B - 2], olds[17], olds[18] = longest, 0, 700
        host, table, _ = make([1] * B, olds, 1, 64, 64, B)
        q = queries(B, 2, 64, "float16", B)
        check(dev, "float16", q, host, table, olds, None, max_kv=longest)
    news = [int(x) for x in np.random.default_rng(5).integers(0, 4, 300)]
    news[7] = 40
    olds = [n + 3 * i % 50 for i, n in enumerate(news)]
    olds[7], olds[299] = 1600, 1400
    host, table, cu = make(news, olds, 1, 64, 64, 7)
    check(dev, "bfloat16", queries(sum(news), 3, 64, "bfloat16"), host, table, olds, cu, max_q=2, max_kv=1600)


def test_very_many_query_heads_and_lengths_beyond_the_table(dev):
    host, table, _ = make([1, 1], [300, 77], 1, 64, 16, 3)
    check(dev, "float16", queries(2, 512, 64, "float16"), host, table, [300, 77], None)
    # kv_lens beyond what the table holds count as that
    table = table[:, :5].copy()
    q = queries(2, 4, 64, "float16")
    check(dev, "float16", q, host, table, [300, 77], None)
    check(dev, "float16", q, host, table, [2 ** 31 - 1, 77], None)


def test_two_streams_at_once(dev):
    """Calls that overlap take workspaces of their own."""
    host, table, _ = make([1], [20000], 2, 128, 64, 21)
    to = lambda a: torch.from_numpy(np.asarray(a)).to(dev)  # noqa: E731
    cache, tab, lens = tuple(to(a) for a in host.arrays()), to(table), to(np.array([20000], np.int32))
    qs = [queries(1, 8, 128, "float16", i).to(dev) for i in range(2)]
    want = [apex4.kv4_attention(q, cache, tab, lens) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(apex4.kv4_attention(qs[i], cache, tab, lens))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_a_workspace_of_the_callers(dev):
    host, table, _ = make([1], [5000], 1, 64, 64, 22)
    to = lambda a: torch.from_numpy(np.asarray(a)).to(dev)  # noqa: E731
    cache, tab, lens = tuple(to(a) for a in host.arrays()), to(table), to(np.array([5000], np.int32))
    q = queries(1, 4, 64, "float16").to(dev)
    need = apex4.kv4_attention_workspace_size(1, 1, 4, 1, 64, 1, tab.shape[1] * 64)
    assert need > 0
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device=dev)          # (NaN wherever it is read unwritten)
    got = apex4.kv4_attention(q, cache, tab, lens, workspace=ws[:need])
    assert torch.equal(got, apex4.kv4_attention(q, cache, tab, lens)) and (ws[need:] == 0xFF).all()
    with pytest.raises(apex4.Apex4Error):
        apex4.kv4_attention(q, cache, tab, lens, workspace=ws[:need - 1])
