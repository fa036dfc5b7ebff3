"""Sizes that the 4-bit cache's calls refuse are refused where the cache is made (CPU)."""
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
