"""What attention over shared prefixes refuses, before anything reaches a GPU."""
import ctypes

import pytest
import torch

from quantized_speculative_decoding_qspec_gb300 import qspec as q

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    return q.load()


def call(lib, cache=(), batch=(), prefixes=(), none=False, **change):
    c = dict(k=FAKE, v=FAKE, k_exp=FAKE, v_exp=FAKE, n_pages=9, heads=2, page=16, dim=64, reserved=0) | dict(cache)
    b = dict(cu=FAKE, kv=FAKE, pages=FAKE, B=4, max_pages=8, max_tok=4, reserved=0, T=16) | dict(batch)
    p = dict(cu=FAKE, len=FAKE, n=2, max_tok=8) | dict(prefixes)
    a = dict(q=FAKE, q_token=256, heads_q=4, scale=1.0, window=0, tree=None, out=FAKE, out_token=256, lse=None, ws=FAKE, ws_bytes=1 << 40)
    a.update(change)
    pre = q.KVPrefixesDesc(*p.values())
    return lib.qspec_kv_attention_shared(ctypes.byref(q.KVCacheDesc(*c.values())), ctypes.byref(q.KVBatchDesc(*b.values())),
                                         None if none else ctypes.byref(pre), *a.values(), None)


@pytest.mark.parametrize("change,code", [
    (dict(none=True), 1), (dict(prefixes=dict(cu=None)), 1), (dict(prefixes=dict(len=None)), 1), (dict(prefixes=dict(n=0)), 1),
    (dict(prefixes=dict(max_tok=0)), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(window=-1), 1), (dict(scale=float("nan")), 1),
    (dict(cache=dict(k=None)), 1), (dict(batch=dict(B=0)), 1), (dict(heads_q=3), 2), (dict(heads_q=258, q_token=1 << 16), 2),
    (dict(tree=FAKE, window=1), 2), (dict(tree=FAKE, batch=dict(max_tok=65, T=100)), 2), (dict(cache=dict(page=8)), 2),
    (dict(batch=dict(B=1025)), 2), (dict(q_token=248), 2), (dict(q=FAKE + 8), 3), (dict(out_token=260), 3), (dict(tree=FAKE + 4), 3),
    (dict(lse=FAKE + 2), 3), (dict(ws=FAKE + 8), 3), (dict(ws=None), 4), (dict(ws_bytes=64), 4)])
def test_arguments(lib, change, code):
    assert call(lib, **change) == code


def test_the_binding_refuses_short_or_wrong_tensors():
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t)  # noqa: E731
    with pytest.raises(ValueError, match="cu_seq holds"):
        q.KVPrefixes(z(3), z(3), 4)
    with pytest.raises(TypeError, match="lengths must be"):
        q.KVPrefixes(z(4), z(3, t=torch.int64), 4)
