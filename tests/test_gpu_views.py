"""Views of a cache's memory keep the cache alive."""
import gc

import pytest
import torch

from kv_cache_decode_kvc_gb300 import kvc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("make", [
    lambda: kvc.KVCache(1, 2, 4, 2, 64, 32), lambda: kvc.KVCache(1, 2, 4, 2, 64, 32, "f32"),
    lambda: kvc.PagedKVCache(1, 6, 16, 2, 3, 4, 2, 64), lambda: kvc.RollingKVCache(1, 2, 4, 2, 128, 32),
    lambda: kvc.QuantKVCache(1, 2, 4, 2, 128, 32), lambda: kvc.QuantKVCache(1, 2, 4, 2, 128, 32, fp8=True)])
def test_views_hold_their_cache(make, monkeypatch):
    # the handle is destroyed when the last view goes, not before (counted on the host: a view
    # without its cache is never read)
    gc.collect()  # caches that earlier tests left
    destroyed = []
    real = kvc.kvc_destroy
    monkeypatch.setattr(kvc, "kvc_destroy", lambda h: (destroyed.append(h), real(h)))
    cache = make()
    views = cache.layer_views(0)
    h = cache.h
    del cache
    gc.collect()
    assert h not in destroyed
    views[0].zero_()
    assert not views[0].float().any()
    last = views[-1][0]
    del views
    gc.collect()
    assert h not in destroyed
    del last
    gc.collect()
    assert destroyed.count(h) == 1
