"""Sizes that the 4-bit cache's calls refuse are refused where the cache is made and the workspace asked for (CPU)."""
import pytest

torch = pytest.importorskip("torch")

from w4a4_group_quantized_amd import apex4  # noqa: E402
from w4a4_group_quantized_amd.attention import KVCache4  # noqa: E402


@pytest.mark.parametrize("bad", [dict(head_dim=96), dict(head_dim=32), dict(head_dim=0), dict(head_dim=512), dict(page=48),
                                 dict(page=0), dict(page=8), dict(page=2048), dict(page=-16), dict(pages=0),
                                 dict(pages=-1), dict(kv_heads=0), dict(kv_heads=1025)])
def test_caches_that_no_call_takes(bad):
    sizes = {**dict(pages=3, kv_heads=2, head_dim=64, page=16), **bad}
    for make in (apex4.kv4_cache, KVCache4):
        with pytest.raises(ValueError):
            make(**sizes, device="cpu")


def test_cache_sizes():
    for D in (64, 128, 256):
        for page in (16, 64, 1024):
            k, ks, v, vs = apex4.kv4_cache(3, 2, D, page, "cpu")
            assert k.shape == (3, 2, page, D // 2) and v.shape == (3, 2, page // 16, 8 * D)
            assert ks.shape == vs.shape == (3, 2, page)


@pytest.mark.parametrize("at", range(1, 7))
@pytest.mark.parametrize("by", [2 ** 32, -2 ** 32, 2 ** 31])
def test_workspace_of_numbers_that_do_not_fit_the_library(monkeypatch, at, by):
    """Taken modulo 2^32 most of them are right arguments; kv4_attention refuses them too."""
    called = []

    class Lib:
        apex4_kv4_attention_workspace_size = staticmethod(lambda *args: called.append(args) or 64)

    monkeypatch.setattr(apex4, "_lib", Lib)
    args = [1, 1, 4, 1, 64, 1, 5000]
    assert apex4.kv4_attention_workspace_size(*args) == 64
    args[at] += by
    with pytest.raises(ValueError):
        apex4.kv4_attention_workspace_size(*args)
    assert len(called) == 1
