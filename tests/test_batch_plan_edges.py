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
