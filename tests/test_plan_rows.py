"""A step's rows are its plan's (CPU)."""
import pytest

torch = pytest.importorskip("torch")

from w4a4_group_quantized_amd import apex4  # noqa: E402
from w4a4_group_quantized_amd.attention import BatchPlan, KVCache4  # noqa: E402


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def test_attention_of_other_rows_than_the_plans(monkeypatch):
    """Fewer rows would end the last sequence early, so that its queries stand at other positions."""
    calls = []
    monkeypatch.setattr(apex4, "kv4_attention", lambda q, *args, **more: calls.append(len(q)) or q)
    cache = KVCache4(4, 2, 64, 16, "cpu")
    plan = BatchPlan(i32([[0, 1], [2, 3]]), i32([20, 5]), i32([0, 4, 7]), page=16, tokens=8)
    for rows in (0, 6, 9):
        with pytest.raises(ValueError):
            cache.attend(torch.zeros((rows, 4, 64), dtype=torch.float16), plan)
    assert cache.attend(torch.zeros((8, 4, 64), dtype=torch.float16), plan).shape == (8, 4, 64) and calls == [8]
