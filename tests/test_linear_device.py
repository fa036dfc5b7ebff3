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

    def dim(self):
        return len(self.shape)

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


def test_the_linear_layers_parts_run_on_their_device(calls, monkeypatch):
    """The quantizers and products that the layer's call is made of, and their forms of other codes."""
    f16, f32 = torch.float16, torch.float32
    for name in ("apex4_quantize_act", "apex4_gemm_w4a4", "apex4_gemm_w4a4_debug", "apex4_gemm_w4a4_noalloc",
                 "apex4_quantize_f8", "apex4_gemm_w4a4_f8", "apex4_quantize_f6", "apex4_gemm_w4a4_f6",
                 "apex4_gemm_workspace_size"):
        value = 0 if "workspace" not in name else 64
        setattr(apex4._lib, name, staticmethod(
            lambda *args, name=name, value=value: calls.append((name, Device.current, args[-1])) or value))
    x, w = Host(3, 256, dtype=f16), Host(256, 256, dtype=f16)
    qa, sa = apex4.quantize_act(x, 128)
    qw, sw = apex4.pack_weight(w, 128)
    y = Host(3, 256, dtype=f16)
    apex4.gemm(qa, sa, 128, qw, sw, 128)
    apex4.gemm(qa, sa, 128, qw, sw, 128, want_psum=True, psum_rows=(0, 1, 2))
    apex4.gemm_noalloc(qa, sa, 128, qw, sw, 128, y16=y)
    a8, w8 = apex4.quantize_f8(x), apex4.quantize_f8(w)
    apex4.gemm_f8(*a8, *w8)
    a6, w6 = apex4.quantize_f6(x), apex4.quantize_f6(w)
    apex4.gemm_f6(*a6, *w6)
    assert len(calls) == 14 and all(c[1] == 1 for c in calls), calls
    assert all(c[2] == 1001 for c in calls if "workspace" not in c[0])
