"""What the page, copy and compacting calls refuse, before anything reaches a GPU."""
import ctypes

import pytest
import torch

from quantized_speculative_decoding_qspec_gb300 import qspec as q

FAKE = 1 << 20          # a 16-byte-aligned stand-in address; never dereferenced (checks fail first)
i32 = torch.int32


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    return q.load()


def pages(lib, **change):
    a = dict(pages=FAKE, room=FAKE, rows=4, max_pages=8, parent=None, keep=FAKE, need=FAKE, new_rows=4, new_max_pages=8, refs=FAKE,
             n_pages=100, page=16, new_pages=FAKE + 4096, new_refs=FAKE, src=FAKE, dst=FAKE, len=FAKE, left=FAKE)
    a.update(change)
    return lib.qspec_kv_pages(*a.values(), None)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), 1), (dict(new_rows=-1), 1), (dict(rows=0, new_rows=0), 1), (dict(refs=None), 1), (dict(new_refs=None), 1),
    (dict(left=None), 1), (dict(n_pages=0), 1), (dict(pages=None), 1), (dict(room=None), 1), (dict(keep=None), 1), (dict(need=None), 1),
    (dict(new_pages=None), 1), (dict(src=None), 1), (dict(dst=None), 1), (dict(len=None), 1), (dict(max_pages=0), 1),
    (dict(new_max_pages=0), 1), (dict(new_pages=FAKE), 1), (dict(new_pages=FAKE + 127), 1), (dict(new_refs=FAKE + 16), 1),
    (dict(page=8), 2), (dict(page=48), 2), (dict(page=256), 2), (dict(rows=1025), 2), (dict(new_rows=1025), 2), (dict(n_pages=1 << 31), 2),
    (dict(max_pages=(1 << 26) + 1, new_pages=FAKE + (1 << 40)), 2), (dict(new_max_pages=(1 << 26) + 1, new_pages=FAKE + (1 << 40)), 2),
    (dict(refs=FAKE + 8, new_refs=FAKE + 8), 3), (dict(new_refs=FAKE + 4096 + 4), 3), (dict(room=FAKE + 2), 3), (dict(parent=FAKE + 1), 3),
    (dict(keep=FAKE + 2), 3), (dict(left=FAKE + 2), 3), (dict(src=FAKE + 2), 3), (dict(new_pages=FAKE + 4098), 3)])
def test_page_tables(lib, change, code):
    assert pages(lib, **change) == code


def cache(**change):
    a = dict(k=FAKE, v=FAKE, k_exp=FAKE, v_exp=FAKE, n_pages=9, heads=2, page=16, dim=64, reserved=0)
    a.update(change)
    return q.KVCacheDesc(*a.values())


@pytest.mark.parametrize("change,code", [
    (dict(k=None), 1), (dict(v_exp=None), 1), (dict(reserved=1), 1), (dict(n_pages=0), 1), (dict(heads=0), 1), (dict(page=24), 2),
    (dict(dim=96), 2), (dict(heads=4097), 2), (dict(k=FAKE + 8), 3)])
def test_caches_of_copies_and_paths(lib, change, code):
    c = cache(**change)
    batch = q.KVBatchDesc(FAKE, FAKE, FAKE, 2, 4, 8, 0, 16)
    assert lib.qspec_kv_copy_pages(ctypes.byref(c), 1, FAKE, FAKE, None, 2, None) == code
    assert lib.qspec_kv_compact(ctypes.byref(c), 1, ctypes.byref(batch), FAKE, FAKE, 8, 1, None) == code


def test_layers_differ_or_are_too_many(lib):
    for change in (dict(n_pages=8), dict(heads=1), dict(page=32), dict(dim=128)):
        arr = (q.KVCacheDesc * 2)(cache(), cache(**change))
        assert lib.qspec_kv_copy_pages(arr, 2, FAKE, FAKE, None, 2, None) == 2
    arr = (q.KVCacheDesc * 65)(*[cache() for _ in range(65)])
    assert lib.qspec_kv_copy_pages(arr, 65, FAKE, FAKE, None, 2, None) == 2
    assert lib.qspec_kv_copy_pages(arr, 0, FAKE, FAKE, None, 2, None) == 1
    assert lib.qspec_kv_copy_pages(None, 1, FAKE, FAKE, None, 2, None) == 1
    assert lib.qspec_kv_copy_pages(arr, 1, None, FAKE, None, 2, None) == 1
    assert lib.qspec_kv_copy_pages(arr, 1, FAKE, FAKE, None, 0, None) == 1
    assert lib.qspec_kv_copy_pages(arr, 1, FAKE, FAKE, FAKE + 2, 2, None) == 3


def test_paths(lib):
    c, batch = cache(), q.KVBatchDesc(FAKE, FAKE, FAKE, 2, 4, 8, 0, 16)
    ref = (ctypes.byref(c), 1, ctypes.byref(batch))
    assert lib.qspec_kv_compact(*ref, None, FAKE, 8, 1, None) == 1
    assert lib.qspec_kv_compact(*ref, FAKE, None, 8, 1, None) == 1
    assert lib.qspec_kv_compact(*ref, FAKE, FAKE, 0, 1, None) == 1
    assert lib.qspec_kv_compact(*ref, FAKE, FAKE, 8, -1, None) == 1
    assert lib.qspec_kv_compact(*ref, FAKE, FAKE, 65, 1, None) == 2
    assert lib.qspec_kv_compact(*ref, FAKE + 2, FAKE, 8, 1, None) == 3
    assert lib.qspec_kv_compact(ref[0], 1, None, FAKE, FAKE, 8, 1, None) == 1


def test_the_binding_refuses_short_tensors():
    z = lambda *s: torch.zeros(*s, dtype=i32)  # noqa: E731
    args = [z(4, 8), z(4), z(3), z(3), z(20), 16, z(3, 8), z(20), z(3), z(3), z(3), z(1)]
    for i, name in ((1, "room"), (2, "keep"), (3, "need"), (7, "new_refs"), (8, "copy_src"), (9, "copy_dst"), (10, "copy_len"), (11, "left")):
        short = list(args)
        short[i] = short[i][:-1]
        with pytest.raises(ValueError, match=name + " holds"):
            q.qspec_kv_pages(*short)
    with pytest.raises(ValueError, match="parent holds"):
        q.qspec_kv_pages(*args, parent=z(2))
    with pytest.raises(TypeError, match="keep must be"):
        q.qspec_kv_pages(*args[:2], z(3).float(), *args[3:])
    with pytest.raises(ValueError, match="dst holds"):
        q.qspec_kv_copy_pages(None, z(3), z(2))
    with pytest.raises(ValueError, match="lengths holds"):
        q.qspec_kv_copy_pages(None, z(3), z(3), lengths=z(2))
    with pytest.raises(ValueError, match="at least one"):
        q.KVLayers([])


def test_a_cache_listed_twice_is_not_compacted(lib):
    batch = q.KVBatchDesc(FAKE, FAKE, FAKE, 2, 4, 8, 0, 16)
    for change in (dict(k=FAKE), dict(v=FAKE)):
        arr = (q.KVCacheDesc * 3)(cache(), cache(k=FAKE * 2, v=FAKE * 3), cache(**dict(dict(k=FAKE * 4, v=FAKE * 5), **change)))
        assert lib.qspec_kv_compact(arr, 3, ctypes.byref(batch), FAKE, FAKE, 8, 1, None) == 1
