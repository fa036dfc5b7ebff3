"""Which device is current when the library is asked (on the CPU: torch's device functions and the library are
replaced): workspace sizes go by the compute units of the current device, launches to it."""
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


@pytest.fixture
def devices(monkeypatch):
    Device.current = 0
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: Device.current)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: Device.current)
    monkeypatch.setattr(torch.cuda, "device", Device)
    return Device


@pytest.mark.parametrize("index", [0, 1])
@pytest.mark.parametrize("fn", ["apex4_experts_workspace_size", "apex4_gemm_e4m3_workspace_size",
                                "apex4_linear_e4m3_workspace_size"])
def test_sizes_are_asked_for_the_tensors_device(devices, monkeypatch, fn, index):
    asked = []

    class Lib:
        pass

    setattr(Lib, fn, staticmethod(lambda *args: asked.append((Device.current, args)) or 77))
    monkeypatch.setattr(apex4, "_lib", Lib)
    assert apex4._size(fn, torch.device("cuda", index), 1, 2, 3) == 77
    assert asked == [(index, (1, 2, 3))] and Device.current == 0


class Host:
    """A host tensor that says it is on a GPU, for what the binding checks before it asks for a size."""
    is_cuda, device = True, torch.device("cuda", 1)

    def __init__(self, *shape, dtype=torch.uint8):
        self.shape, self.dtype = torch.Size(shape), dtype

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True


def test_the_calls_ask_that_way(devices, monkeypatch):
    asked = []

    class Stop(Exception):
        pass

    def answer(*_):
        asked.append(Device.current)
        raise Stop

    class Lib:
        apex4_experts_workspace_size = apex4_gemm_e4m3_workspace_size = apex4_linear_e4m3_workspace_size = \
            staticmethod(answer)

    monkeypatch.setattr(apex4, "_lib", Lib)
    f16, f32, i32 = torch.float16, torch.float32, torch.int32
    y = Host(3, 256, dtype=f16)
    with pytest.raises(Stop):
        apex4.experts(Host(3, 256, dtype=f16), Host(3, 2, dtype=i32), Host(3, 2, dtype=f32), Host(4, 256, 128),
                      Host(4, 256, 2, dtype=f32), Host(4, 256, 64), Host(4, 256, 1, dtype=f32), y16=y)
    with pytest.raises(Stop):
        apex4.gemm_e4m3(Host(3, 256), Host(3, 2, dtype=f32), Host(256, 256), Host(2, 2, dtype=f32), y=y)
    with pytest.raises(Stop):
        apex4.linear_e4m3(Host(3, 256, dtype=f16), Host(256, 256), Host(2, 2, dtype=f32), y=y)
    assert asked == [1, 1, 1]


def test_experts_are_packed_on_their_device(devices, monkeypatch):
    from w4a4_group_quantized_amd.sparse import W4A4Experts
    packed = []

    def pack(w, group):
        packed.append(Device.current)
        return torch.zeros(w.shape[0], 1, dtype=torch.uint8), torch.zeros(w.shape[0], 1)

    class OnDevice1(torch.Tensor):
        device = property(lambda self: torch.device("cuda", 1))

    monkeypatch.setattr(apex4, "pack_weight", pack)
    with pytest.raises(ValueError):        # the packed tensors are on the host
        W4A4Experts.from_weights(torch.zeros(2, 4, 8).as_subclass(OnDevice1), torch.zeros(2, 4, 2).as_subclass(OnDevice1))
    assert packed == [1, 1] and Device.current == 0


@pytest.mark.parametrize("bad", [dict(n_group=2 ** 32 + 8, topk_group=4), dict(n_group=8, topk_group=2 ** 32 + 4),
                                 dict(group_top=2 ** 32 + 1), dict(group_top=-2 ** 32 + 2), dict(k=2 ** 33 + 6),
                                 dict(k=-2 ** 32 + 6)])
def test_route_refuses_numbers_that_do_not_fit_the_library(devices, monkeypatch, bad):
    """Taken modulo 2^32 each of them is a right argument."""
    called = []

    class Lib:
        apex4_route = staticmethod(lambda *args: called.append(args) or 0)

    class Logits(Host):
        def data_ptr(self):
            return 0x10000

    monkeypatch.setattr(apex4, "_lib", Lib)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0)
    args = dict(k=6) | bad
    out = Logits(4, args["k"], dtype=torch.int32), Logits(4, args["k"], dtype=torch.float32)
    with pytest.raises(ValueError, match="32 bits"):
        apex4.route(Logits(4, 64, dtype=torch.float32), out=out, **args)
    assert not called
