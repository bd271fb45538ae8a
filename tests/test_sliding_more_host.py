"""Classes of sliding-window serving without a GPU: what they hold and what they refuse."""
import gc
import weakref

import pytest

from test_ops_host import lib as built  # noqa: F401  (a fixture)

torch = pytest.importorskip("torch")


@pytest.fixture
def cache_py(built, monkeypatch):  # noqa: F811
    from quantized_kv_cache_07_gb300 import cache
    monkeypatch.setattr(cache, "_require_cuda", lambda: None)
    return cache


def test_a_descriptor_holds_its_buffers(cache_py):
    """What a list of caches points at lives as long as the list, as a rotary table's descriptor holds its table."""
    lib = cache_py._lib
    c = cache_py.KVCache(3, 2, 4, 4, window=16, window_batch=2, channel_factor=[[1.0] * 128] * 2, device="cpu")
    tensors = (c.k_codes, c.v_codes, c.meta, c.k_window, c.v_window, c.channel_factor)
    storages = [weakref.ref(t) for t in tensors]
    layers = lib.CacheList([c.desc])
    del c, tensors
    gc.collect()
    assert all(s() is not None for s in storages)
    assert layers.array[0].k_codes == storages[0]().data_ptr()
    del layers
    gc.collect()
    assert all(s() is None for s in storages)


def test_pages_refuse_rings_of_fewer_rows(cache_py):
    """An update that forks rows would leave its tables changed and its rings not: refused when the pages are made."""
    make = lambda rows: cache_py.KVCache(8, 1, 8, 8, window=16, window_batch=rows, device="cpu")
    with pytest.raises(ValueError):
        cache_py.Pages([make(4), make(3)], 4, 8)
    pages = cache_py.Pages([make(4), make(7)], 4, 8)
    assert pages.table.shape == (4, 8)
    cache_py.Pages([cache_py.KVCache(8, 1, 8, 8, device="cpu")], 4, 8)  # no rings: any batch


def test_pages_refuse_caches_of_two_devices(cache_py):
    one, other = (cache_py.KVCache(8, 1, 8, 8, device="cpu") for _ in range(2))
    cache_py.Pages([one, other], 2, 4)
    other.k_codes = other.k_codes.to("meta")
    with pytest.raises(ValueError):
        cache_py.Pages([one, other], 2, 4)
