"""BatchPlan: where a step's tokens stand and are kept, against a loop over the sequences."""
import pytest

torch = pytest.importorskip("torch")

from w4a4_group_quantized_amd.attention import BatchPlan  # noqa: E402


def expected(table, kv_lens, cu, page, tokens):
    positions, slots = [0] * tokens, [-1] * tokens
    for b, kv in enumerate(kv_lens):
        for row in range(cu[b], min(cu[b + 1], tokens)):
            at = kv - (cu[b + 1] - row)
            if 0 <= at < len(table[b]) * page:
                positions[row] = at
                if table[b][at // page] >= 0:
                    slots[row] = table[b][at // page] * page + at % page
    return positions, slots


@pytest.mark.parametrize("first,behind", [(0, 0), (0, 5), (3, 0), (4, 7)])
@pytest.mark.parametrize("news,kv_lens", [([3, 1, 2], [3, 40, 17]), ([0, 4, 0], [9, 4, 0]), ([5, 1, 1], [2, 64, 65]),
                                          ([1, 1, 1], [1, 16, 33])])
def test_positions_and_slots(first, behind, news, kv_lens):
    """Padding on both sides, empty sequences, more queries than tokens, a length beyond the table, no page."""
    table = [[5, 2, 9, 0], [1, -1, 3, 8], [7, 6, 4, 10]]
    cu = [first]
    for n in news:
        cu.append(cu[-1] + n)
    tokens = cu[-1] + behind
    as_int = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    plan = BatchPlan(as_int(table), as_int(kv_lens), as_int(cu), page=16, tokens=tokens)
    assert (plan.positions.tolist(), plan.slots.tolist()) == expected(table, kv_lens, cu, 16, tokens)
    if news == [1, 1, 1] and first == behind == 0:
        one = BatchPlan(as_int(table), as_int(kv_lens), page=16)
        assert torch.equal(one.positions, plan.positions) and torch.equal(one.slots, plan.slots)


def test_rows_of_a_step_are_given_with_cu_q():
    table = torch.zeros((2, 4), dtype=torch.int32)
    with pytest.raises(ValueError):
        BatchPlan(table, torch.ones(2, dtype=torch.int32), torch.arange(3, dtype=torch.int32), page=16)
