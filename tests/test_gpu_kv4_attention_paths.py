"""apex4_kv4_attention through every kernel instance that a call's sizes can choose (attention_rows.cut says which;
tests/test_attention_cut.py holds it against the library's rule): all rows against attention in 64 bits, some of
them against the bound that follows each token's weight."""
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


def make(olds, heads, D, page, seed, extra=2):
    """A filled cache on the host and a shuffled table (unused entries are not pages)."""
    rng = np.random.default_rng(seed)
    need = [-(-int(n) // page) for n in olds]
    host = ref.Cache(sum(need) + extra, heads, page, D, seed + 1)
    order, at = rng.permutation(sum(need) + extra), 0
    table = np.full((len(olds), max(1, max(need))), -7, np.int32)
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return host, table


def way(q, host, olds, cu, max_q, max_kv, window=0):
    T, Hq, D = q.shape
    return cut(T, len(olds), Hq, host.kc.shape[1], D, max_q, max_kv, window,
               torch.cuda.get_device_properties(0).multi_processor_count)


def run(dev, q, host, table, olds, cu, **args):
    """Outputs of the call, which writes between guard rows; q is a part of wider rows."""
    to = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(dev)  # noqa: E731
    cache = tuple(torch.from_numpy(a).to(dev) for a in host.arrays())
    T, H, D = q.shape
    wide = torch.zeros((T, H + 3, D), dtype=q.dtype, device=dev)
    wide[:, 1:H + 1] = q.to(dev)
    out, lse = torch.full((T + 2, H, D), 7.0, dtype=q.dtype, device=dev), torch.full((T + 2, H), 7.0, device=dev)
    apex4.kv4_attention(wide[:, 1:H + 1], cache, to(table), to(olds), None if cu is None else to(cu), want_lse=True,
                        out=out[1:-1], lse=lse[1:-1], **args)
    torch.cuda.synchronize()
    assert (out[[0, -1]] == 7).all() and (lse[[0, -1]] == 7).all()
    return out[1:-1].double().cpu().numpy(), lse[1:-1].double().cpu().numpy()


def check(dev, dtype, q, host, table, olds, cu, max_q, max_kv, some=24, adds=None, every=True, **args):
    """Every row (unless `every` is false) within ref.attention's bound, `some` of them within
    attention_rows', which follow `adds` additions by one wave."""
    got, got_lse = run(dev, q, host, table, olds, cu, max_q=max_q, max_kv=max_kv, **args)
    numbers = q.double().numpy()
    ends = np.arange(len(olds) + 1) if cu is None else np.asarray(cu)
    owned = np.zeros(len(q), bool)
    owned[ends[0]:ends[-1]] = True
    if every:
        want, lse, bound, lse_bound, _ = ref.attention(numbers, dtype, host, table, olds, cu, **args)
        assert (got[~owned] == 7).all() and (got_lse[~owned] == 7).all()
        nan, mine = np.isnan(want).any(-1), np.broadcast_to(owned[:, None], want.shape[:2])
        assert np.isnan(got[nan & mine]).all()             # (what is not finite reaches all of a row)
        over = ref.off(got, want, bound, dtype) & (mine & ~nan)[..., None]
        assert not over.any(), (np.argwhere(over)[:4], np.abs(got - want)[over].max(), bound[over][:4])
        none = np.isneginf(lse) & mine
        assert (got[none] == 0).all() and np.isneginf(got_lse[none]).all()
        live = mine & ~nan & np.isfinite(lse)
        assert (np.abs(got_lse[live] - lse[live]) <= lse_bound[live]).all()
    rng = np.random.default_rng(1)
    first, last = int(ends[0]), int(ends[-1]) - 1
    rows = sorted({(int(t), int(h)) for t, h in zip(rng.integers(first, last + 1, some), rng.integers(0, q.shape[1], some))}
                  | {(first, 0), (last, q.shape[1] - 1)})
    rows = [r for r in rows if np.isfinite(numbers[r]).all()]
    o, lse, bound, lse_bound = attention_rows(numbers, dtype, host, table, olds, cu, rows, run=adds, **args)
    for at, (t, h) in enumerate(rows):
        if np.isnan(o[at]).any():
            continue
        over = ref.off(got[t, h], o[at], bound[at], dtype)
        assert not over.any(), (t, h, got[t, h][over][:4], o[at][over][:4], bound[at][over][:4])
        assert got_lse[t, h] == lse[at] or abs(got_lse[t, h] - lse[at]) <= lse_bound[at], (t, h)


def queries(T, H, D, dtype, seed=0):
    return (1.3 * torch.randn((T, H, D), generator=torch.Generator().manual_seed(seed))).to(getattr(torch, dtype))


HEADS = [(64, 64, 8), (128, 64, 8), (256, 32, 8)]                 # D, query and key heads


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("D,Hq,Hkv", HEADS)
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 150), (False, 0)])
def test_prompt(dev, dtype, D, Hq, Hkv, causal, window):
    """One prompt, and two of one length: neither rows nor tokens fill their tiles."""
    for news, olds, page in (([803], [937], 64), ([405, 405], [405, 611], 16)):
        host, table = make(olds, Hkv, D, page, D + window)
        q = queries(sum(news), Hq, D, dtype, window)
        cu = np.concatenate(([0], np.cumsum(news)))
        assert way(q, host, olds, cu, max(news), max(olds), window) == dict(
            kernel="rows", rt=1 if D == 256 else 2, uneven=False, share=False, deep=False, sorted=False)
        check(dev, dtype, q, host, table, olds, cu, max(news), max(olds), causal=causal, window=window)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 16, 4), (128, 16, 4), (256, 8, 4)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 90), (False, 0)])
def test_prompts_among_short_sequences(dev, dtype, D, Hq, Hkv, causal, window):
    """Uneven batches, with padding before the first sequence and behind the last, and sequences of none."""
    rng = np.random.default_rng(D)
    news = rng.integers(0, 3, 70)
    news[[3, 20, 64]] = 900, 30, 811
    olds = news + rng.integers(0, 200, 70)
    olds[[3, 5]] = 900, 0
    host, table = make(olds, Hkv, D, 16, D + 1)
    cu = np.concatenate(([0], np.cumsum(news))) + 21
    q = queries(int(cu[-1]) + 9, Hq, D, dtype, 2)
    w = way(q, host, olds, cu, 900, int(olds.max()), window)
    assert w["kernel"] == "rows" and w["uneven"] and w["rt"] == (1 if D == 256 else 2)
    check(dev, dtype, q, host, table, olds, cu, 900, int(olds.max()), causal=causal, window=window)


@pytest.mark.parametrize("D,Hq,Hkv", HEADS)
def test_prompt_with_pages_that_are_none_and_numbers_that_are(dev, D, Hq, Hkv):
    """Pages outside the cache, NaN scales behind the sequence, in a key and in a value, queries that are not
    finite, tiny or huge (bf16): each shows in the rows that see it."""
    T, kv = 803, 900
    host, table = make([kv], Hkv, D, 16, 9)
    used = np.zeros(host.ks.shape[0::2], bool)
    used[table[0, np.arange(kv) // 16], np.arange(kv) % 16] = True
    for s in (host.ks, host.vs):
        s.transpose(0, 2, 1)[~used] = np.nan
    table[0, [3, 20, 21, 50]] = -1, len(host.kc), 2 ** 31 - 1, -2 ** 31
    host.ks[table[0, 890 // 16], 1, 890 % 16] = np.nan
    q = queries(T, Hq, D, "bfloat16", 5)
    q[:, 1] *= 2.0 ** -40
    q[:, 2] *= 2.0 ** 20
    host.ks[:, 0] *= np.float32(2.0 ** -12)
    q[:, 3] = 0
    q[100, 5, 7], q[101, Hq - 1, D - 1], q[102, 6, 0] = float("nan"), float("inf"), float("-inf")
    clean = q.clone()
    clean[100, 5, 7] = clean[101, Hq - 1, D - 1] = clean[102, 6, 0] = 0
    args = (host, table, [kv], [0, T])
    assert way(q, host, [kv], [0, T], T, kv)["kernel"] == "rows"
    got, _ = run(dev, q, *args, max_q=T, max_kv=kv)
    other, _ = run(dev, clean, *args, max_q=T, max_kv=kv)
    mine = np.zeros(got.shape[:2], bool)
    mine[100, 5] = mine[101, Hq - 1] = mine[102, 6] = True
    assert np.isnan(got[mine]).all() and np.array_equal(got[~mine], other[~mine], equal_nan=True)
    check(dev, "bfloat16", clean, *args, T, kv)
    host.vs[table[0, 500 // 16], 2, 500 % 16] = np.nan
    got, _ = run(dev, clean, *args, max_q=T, max_kv=kv)
    mine[:] = False
    mine[500 - (kv - T):, 2 * (Hq // Hkv):3 * (Hq // Hkv)] = True
    assert np.isnan(got[mine]).all() and np.array_equal(got[~mine], other[~mine], equal_nan=True)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,Hkv,share,news,window", [(64, 8, 2, 1, 0), (66, 8, 1, 1, 0), (256, 2, 2, 1, 0), (66, 8, 2, 1, 1400),
                                                     (24, 8, 8, 12, 0)])
def test_longest_first(dev, dtype, D, B, Hkv, share, news, window):
    """Decoding sequences (and short drafts, several row tiles each) in the order of their lengths: many of one
    length, some empty."""
    if news > 1 and D == 256:
        B, news = 40, 3                                    # (row tiles of 16, not 32)
    rng = np.random.default_rng(B + D)
    olds = rng.choice([0, 12, 300, 700, 701, 1000, 1500], B)
    olds[[0, B - 1]] = 1700, 1700
    count = rng.integers(0, news + 1, B) if news > 1 else np.ones(B, int)
    count[[1, B - 1]] = news
    if news > 1:
        count[2:B - 1] = np.maximum(count[2:B - 1], 2 * news // 3)
    # (sequences share the pages of four)
    host, four = make([1700] * 4, Hkv, D, 64, B)
    table = four[np.arange(B) % 4]
    cu = np.concatenate(([0], np.cumsum(count)))
    q = queries(int(cu[-1]), Hkv * share, D, dtype, B)
    w = way(q, host, olds, cu, news, 1700, window)
    assert w["kernel"] == "few" and w["sorted"] and not w["uneven"] and w["rt"] == (2 if news > 1 and D < 256 else 1)
    check(dev, dtype, q, host, table, olds, None if news == 1 else cu, news, 1700, window=window)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("deep", [True, False])
@pytest.mark.parametrize("D,rt", [(64, 1), (64, 2), (128, 1), (128, 2), (256, 1)])
def test_shared_row_tiles(dev, dtype, D, rt, deep):
    """Row tiles in parts, joined by one wave a row or by 16."""
    news, olds = ([1, 1, 1], [0, 77, 3100]) if rt == 1 else ([21, 1, 9], [2500, 1, 400])
    if not deep:
        olds = [min(o, 2000) for o in olds]
    host, table = make(olds, 2, D, 32, D + rt)
    q = queries(sum(news), 8, D, dtype, 3)
    cu = np.concatenate(([0], np.cumsum(news)))
    w = way(q, host, olds, cu, max(news), max(olds))
    assert w["kernel"] == "few" and w["share"] and w["rt"] == rt and w["deep"] == deep
    check(dev, dtype, q, host, table, olds, cu, max(news), max(olds))


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_several_units_a_workgroup(dev, dtype, D):
    """More units than workgroups: a workgroup ends one row tile, has whole ones and begins another."""
    olds = list(np.random.default_rng(D).integers(0, 3100, 20))
    olds[4], olds[5] = 0, 3100
    host, four = make([3100] * 2, 8, D, 64, D)
    table = four[np.arange(20) % 2]
    q = queries(20, 16, D, dtype, 8)
    w = way(q, host, olds, None, 1, 3100)
    assert w["share"] and not w["deep"]
    check(dev, dtype, q, host, table, olds, None, 1, 3100)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_whole_row_tiles(dev, dtype, D):
    """Few tokens: no workgroup shares a tile, two row tiles of 16 a wave or one."""
    for news, olds in (([1, 1], [900, 3]), ([40, 3], [800, 3]), ([70, 1, 0], [70, 900, 12])):
        host, table = make(olds, 2, D, 16, D)
        q = queries(sum(news), 6, D, dtype, 4)
        cu = np.concatenate(([0], np.cumsum(news)))
        w = way(q, host, olds, cu, max(news), max(olds))
        assert w["kernel"] == "few" and not w["share"] and not w["sorted"]
        check(dev, dtype, q, host, table, olds, cu, max(news), max(olds))


@pytest.mark.parametrize("dtype,D,Hq,kv", [("float16", 128, 8, 131071), ("bfloat16", 64, 3, 131072), ("float16", 256, 1, 100003)])
def test_one_very_long_sequence(dev, dtype, D, Hq, kv):
    """Each wave adds 64 to 128 tokens, the join up to 512 parts."""
    host, table = make([kv], 1, D, 256, 11)
    host.ks *= np.float32(1.7)                               # (some tokens well above the others)
    q = queries(1, Hq, D, dtype, 6)
    assert way(q, host, [kv], None, 1, kv)["deep"]
    check(dev, dtype, q, host, table, [kv], None, 1, kv, adds=128 + 8 * 512, every=False)


def test_prompt_behind_a_long_context(dev):
    """One wave adds all of 30011 tokens."""
    T, kv = 800, 30011
    host, table = make([kv], 2, 64, 128, 12)
    q = queries(T, 64, 64, "float16", 7)
    assert way(q, host, [kv], [0, T], T, kv)["kernel"] == "rows"
    check(dev, "float16", q, host, table, [kv], [0, T], T, kv, every=False)
