"""KVCache keeps its tensors' addresses: neither may change behind a call. On
the CPU, with the checks of the tensors' device left out."""
import pytest
import torch

import bit_gemv_amd as bg


@pytest.fixture(params=[True, False])
def cache(request, monkeypatch):
    monkeypatch.setattr(bg, "_need", lambda *a: None)
    monkeypatch.setattr(bg, "_on", lambda *a: None)
    return bg.KVCache.empty(2, 16, 1, 64, symmetric=request.param, device="cpu")


def _calls(cache):
    x = torch.zeros((1, 1, 64))
    batch = torch.zeros((1, 1), dtype=torch.int32), torch.ones(1, dtype=torch.int32), torch.tensor([0, 1], dtype=torch.int32)
    return (lambda: bg.kv_cache_write(x, x, cache, *batch), lambda: bg.kv_cache_read(cache, *batch, rows=1),
            lambda: bg.paged_attention(x.bfloat16(), cache, *batch))


@pytest.mark.parametrize("name", ["k_codes", "v_codes", "k_scales", "v_scales", "k_zeros", "v_zeros", "heads", "head_dim",
                                  "pages", "page_size", "bits", "symmetric", "device"])
def test_nothing_can_be_assigned(cache, name):
    was = getattr(cache, name)
    with pytest.raises(AttributeError, match=name):
        setattr(cache, name, was)
    with pytest.raises(AttributeError, match=name):
        delattr(cache, name)
    assert getattr(cache, name) is was


@pytest.mark.parametrize("name", ["k_codes", "v_codes", "k_scales", "v_scales", "k_zeros", "v_zeros"])
def test_tensors_that_moved_are_refused(cache, name):
    t = getattr(cache, name)
    if t is None:
        return
    t.set_(t.clone())
    for call in _calls(cache):
        with pytest.raises(ValueError, match="moved"):
            call()


def test_freed_storage_is_refused(cache):
    cache.k_codes.untyped_storage().resize_(0)
    for call in _calls(cache):
        with pytest.raises(ValueError, match="moved"):
            call()


def test_contents_may_change(cache):
    cache.k_codes.zero_()
    cache.k_scales.copy_(torch.rand(2, 1, 16))
    assert cache._live() == cache._ref


def test_a_programs_own_attributes(cache):
    cache.table = 3
    assert cache.table == 3
    del cache.table

    class Named(bg.KVCache):
        def __init__(self, *args):
            super().__init__(*args)
            self.name = "layer 1"

    c = Named(cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales, cache.k_zeros, cache.v_zeros, 64, 8)
    assert c.name == "layer 1" and c._live() == c._ref
