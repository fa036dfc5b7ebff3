"""BatchPlan: padded decoding batches (CPU)."""
import pytest

torch = pytest.importorskip("torch")

from w4a4_group_quantized_amd.attention import BatchPlan  # noqa: E402


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def test_one_token_a_sequence_and_padding_behind():
    """More rows than sequences: attention is told where the sequences' rows end."""
    plan = BatchPlan(i32([[4, -1], [2, 7]]), i32([5, 18]), page=16, tokens=5)
    assert plan.positions.tolist() == [4, 17, 0, 0, 0] and plan.slots.tolist() == [68, 7 * 16 + 1, -1, -1, -1]
    assert plan.tokens == 5 and plan.cu_q.tolist() == [0, 1, 2] and plan.cu_q.dtype == torch.int32 and plan.max_q == 1
    plan = BatchPlan(i32([[4, -1], [2, 7]]), i32([5, 18]), page=16, tokens=2)
    assert plan.cu_q is None and plan.max_q is None


def test_fewer_rows_than_sequences():
    with pytest.raises(ValueError):
        BatchPlan(i32([[4, -1], [2, 7]]), i32([5, 18]), page=16, tokens=1)


@pytest.mark.parametrize("cu", [None, [0], [2]])
def test_no_sequences(cu):
    """An idle step: rows of padding only."""
    none = torch.zeros((0, 3), dtype=torch.int32)
    for tokens in (0, 4):
        plan = BatchPlan(none, i32([]), None if cu is None else i32(cu), page=16, tokens=tokens)
        assert plan.positions.tolist() == [0] * tokens and plan.slots.tolist() == [-1] * tokens
        assert plan.positions.dtype == plan.slots.dtype == torch.int64
        assert tokens == 0 or plan.cu_q is not None


def test_refusals():
    """What the cache or the attention would refuse only after the tokens are stored, or index out of range."""
    table, lens, cu = i32([[4, -1], [2, 7]]), i32([5, 18]), i32([0, 1, 2])
    for bad in (dict(page=0), dict(page=8), dict(page=24), dict(page=2048), dict(table=table[0]), dict(table=table.long()),
                dict(table=table[:, :0]), dict(kv_lens=lens[:1]), dict(kv_lens=lens.long()), dict(cu_q=cu[:2]),
                dict(cu_q=cu.long()), dict(tokens=-1), dict(kv_lens=lens.to("meta"))):
        with pytest.raises(ValueError):
            BatchPlan(**{**dict(table=table, kv_lens=lens, cu_q=cu, page=16, tokens=2), **bad})


def test_parts_of_wider_tables():
    """The first columns of a table with room for more, every other length: as copies of them."""
    wide = i32([[4, -1, 9], [2, 7, 9]])
    lens, cu = i32([5, 0, 18, 0]), i32([0, 9, 1, 9, 2])
    plan = BatchPlan(wide[:, :2], lens[::2], cu[::2], page=16, tokens=2)
    want = BatchPlan(wide[:, :2].contiguous(), i32([5, 18]), i32([0, 1, 2]), page=16, tokens=2)
    for name in ("table", "kv_lens", "cu_q", "positions", "slots"):
        assert torch.equal(getattr(plan, name), getattr(want, name)) and getattr(plan, name).is_contiguous()
