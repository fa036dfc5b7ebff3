"""Which device is current when a linear layer reaches the library (on the CPU: torch's device functions and the
library are replaced): launches go to the current device, the layer's tensors may be on another one."""
import pytest

torch = pytest.importorskip("torch")

from w4a4_group_quantized_amd import apex4  # noqa: E402


class Device:
    """In place of torch.cuda.device."""
    current = 0

    def __init__(self, device):
        self.index = torch.device(device).index

    def __enter__(self):
        self.before, Device.current = Device.current, self.index

    def __exit__(self, *_):
        Device.current = self.before


class Host:
    """A host tensor that says it is on GPU 1."""
    is_cuda, device = True, torch.device("cuda", 1)

    def __init__(self, *shape, dtype=torch.uint8):
        self.shape, self.dtype = torch.Size(shape), dtype

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 0x10000


@pytest.fixture
def calls(monkeypatch):
    Device.current = 0
    seen = []

    class Lib:
        pass

    def record(name, result):
        return staticmethod(lambda *args: seen.append((name, Device.current, args[-1])) or result)

    setattr(Lib, "apex4_linear_w4a4", record("apex4_linear_w4a4", 0))
    setattr(Lib, "apex4_linear_workspace_size", record("size", 512))
    setattr(Lib, "apex4_pack_weight", record("apex4_pack_weight", 0))

    class Stream:
        cuda_stream = 1001

    monkeypatch.setattr(apex4, "_lib", Lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: Device.current, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: Stream)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None: Host(
        *((shape,) if isinstance(shape, int) else shape), dtype=dtype))
    return seen


def test_a_linear_layer_runs_and_packs_on_its_device(calls):
    qw, sw = apex4.pack_weight(Host(256, 256, dtype=torch.float16), 128)
    apex4.linear(Host(3, 256, dtype=torch.float16), 128, qw, sw, 128)
    assert [c[0] for c in calls] == ["apex4_pack_weight", "size", "apex4_linear_w4a4"]
    assert all(c[1] == 1 for c in calls) and Device.current == 0
    assert all(c[2] == 1001 for c in calls if c[0] != "size")            # the device's own stream
