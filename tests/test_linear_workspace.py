"""W4A4Linear's calls share no workspace (on the CPU: the library's call is replaced)."""
import pytest

torch = pytest.importorskip("torch")

from w4a4_group_quantized_amd import apex4  # noqa: E402
from w4a4_group_quantized_amd.linear import W4A4Linear  # noqa: E402


class OnGpu(torch.Tensor):
    """A host tensor that says it is on a GPU."""
    is_cuda = property(lambda self: True)


def test_calls_in_flight_have_workspaces_of_their_own(monkeypatch):
    """Calls of one row count, as two streams or two captured graphs have them in flight at once."""
    given = []

    def linear(x, ga, qw, sw, gw, *, y16=None, workspace=None):
        given.append(workspace)                            # (None: the call allocates its own)
        return torch.zeros((x.shape[0], qw.shape[0]), dtype=torch.float16)

    monkeypatch.setattr(apex4, "linear", linear)
    monkeypatch.setattr(apex4, "linear_workspace_size", lambda *_: 4096)
    m = W4A4Linear(torch.zeros((256, 128), dtype=torch.uint8).as_subclass(OnGpu), torch.ones((256, 2)), 128)
    for _ in range(3):
        assert m(torch.zeros((5, 256), dtype=torch.float16)).shape == (5, 256)
    places = [w.data_ptr() for w in given if w is not None]
    assert len(given) == 3 and len(set(places)) == len(places)
