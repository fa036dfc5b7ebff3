"""Which device is current when the rotary, cache and attention calls reach the library (on the CPU: torch's
device functions and the library are replaced)."""
import pytest

torch = pytest.importorskip("torch")

from w4a4_group_quantized_amd import apex4  # noqa: E402


class Device:
    """In place of torch.cuda.device."""
    current = 0

    def __init__(self, index):
        self.index = index if isinstance(index, int) else torch.device(index).index

    def __enter__(self):
        self.before, Device.current = Device.current, self.index

    def __exit__(self, *_):
        Device.current = self.before


class Host:
    """A host tensor that says it is on GPU 1."""
    device = torch.device("cuda", 1)
    is_cuda = True

    def __init__(self, *shape, dtype=torch.float16):
        self.shape, self.dtype = torch.Size(shape), dtype

    def get_device(self):
        return 1

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self):
        out = [1]
        for n in reversed(self.shape[1:]):
            out.insert(0, out[0] * n)
        return tuple(out)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000

    def new_empty(self, shape):
        return Host(*shape, dtype=self.dtype)


@pytest.fixture
def calls(monkeypatch):
    Device.current = 0
    seen = []

    class Lib:
        pass

    def record(name, result):
        return staticmethod(lambda *args: seen.append((name, Device.current, args[-1])) or result)

    for name in ("apex4_rope", "apex4_kv4_append", "apex4_kv4_read", "apex4_kv4_attention"):
        setattr(Lib, name, record(name, 0))
    setattr(Lib, "apex4_kv4_attention_workspace_size", record("size", 512))
    monkeypatch.setattr(apex4, "_lib", Lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: Device.current, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None: Host(
        *((shape,) if isinstance(shape, int) else shape), dtype=dtype))
    return seen


def test_calls_run_on_the_tensors_device(calls):
    cache = (Host(4, 2, 16, 32, dtype=torch.uint8), Host(4, 2, 16, dtype=torch.float32),
             Host(4, 2, 1, 512, dtype=torch.uint8), Host(4, 2, 16, dtype=torch.float32))
    x, k = Host(3, 4, 64), Host(3, 2, 64)
    slots, freq = Host(3, dtype=torch.int64), Host(32, dtype=torch.float64)
    apex4.rope(x, slots, freq)
    apex4.kv4_append(cache, k, k, slots, positions=slots, inv_freq=freq, q=x)
    apex4.kv4_read(cache, slots)
    apex4.kv4_attention(x, cache, Host(3, 2, dtype=torch.int32), Host(3, dtype=torch.int32))
    assert [c[0] for c in calls] == ["apex4_rope", "apex4_kv4_append", "apex4_kv4_read", "size", "apex4_kv4_attention"]
    assert all(c[1] == 1 for c in calls) and Device.current == 0
    assert all(c[2] == 1001 for c in calls if c[0] != "size")            # the device's own stream
