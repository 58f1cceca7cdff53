"""A step whose last rows have ended asks for no page copies: the copying call takes none as it is (no GPU)."""
import ctypes

import pytest
import torch

from quantized_speculative_decoding_qspec_gb300 import qspec as q

FAKE = 1 << 20          # a 16-byte-aligned stand-in address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    return q.load()


def cache(**change):
    a = dict(k=FAKE, v=FAKE, k_exp=FAKE, v_exp=FAKE, n_pages=9, heads=2, page=16, dim=64, reserved=0)
    a.update(change)
    return q.KVCacheDesc(*a.values())


def test_no_pairs_without_arrays(lib):
    c = cache()
    assert lib.qspec_kv_copy_pages(ctypes.byref(c), 1, None, None, None, 0, None) == 0
    # what else is checked still is; pairs need their arrays, and a number of them
    assert lib.qspec_kv_copy_pages(None, 1, None, None, None, 0, None) == 1
    bad = cache(page=24)
    assert lib.qspec_kv_copy_pages(ctypes.byref(bad), 1, None, None, None, 0, None) == 2
    assert lib.qspec_kv_copy_pages(ctypes.byref(c), 1, None, None, None, -1, None) == 1
    assert lib.qspec_kv_copy_pages(ctypes.byref(c), 1, None, FAKE, None, 1, None) == 1
    assert lib.qspec_kv_copy_pages(ctypes.byref(c), 1, FAKE, FAKE, None, 0, None) == 1


class Device(torch.Tensor):
    """A tensor that says it is on the GPU; its address is never used."""
    is_cuda = property(lambda self: True)


def test_the_binding_hands_on_empty_arrays(lib, monkeypatch):
    monkeypatch.setattr(q, "_stream", lambda stream: None)
    none = torch.zeros(4, dtype=torch.int32)[:0].as_subclass(Device)
    layers = q.KVLayers.__new__(q.KVLayers)
    layers.arr = (q.KVCacheDesc * 2)(cache(), cache())
    layers.n, layers.page, layers.ref = 2, 16, ctypes.addressof(layers.arr)
    q.qspec_kv_copy_pages(layers, none, none, lengths=none)
    q.qspec_kv_copy_pages(layers, none, none)
    q.qspec_kv_copy_pages(layers, none, torch.zeros(4, dtype=torch.int32).as_subclass(Device))   # (room for more pairs)
