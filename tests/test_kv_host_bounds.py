"""Refusals around the edges of the rotary, cache, attention and logits calls (no GPU)."""
import ctypes
import itertools

import pytest
import torch

from quantized_speculative_decoding_qspec_gb300 import qspec as q

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    return q.load()


def test_rotary_refuses_outputs_that_overlap(lib):
    """Every layout of a few tokens and heads, against the rows' addresses.  (The positions' address is misaligned,
    which is looked at afterwards: no call reaches a GPU.)"""
    plan = ctypes.byref(q.RotaryPlan(FAKE, 8, 0, 1.0, 0))
    D = 8

    def call(T, H, token, head):
        return lib.qspec_rotary(FAKE, 0, 0, FAKE + 2, T, H, D, plan, 0, FAKE, token, head, None)

    seen = set()
    for T, H, token, head in itertools.product((1, 2, 3, 5), (1, 2, 3, 4), range(0, 80, 8), range(0, 80, 8)):
        rows = [t * token + h * head for t in range(T) for h in range(H)]
        overlap = any(abs(a - b) < D for a, b in itertools.combinations(rows, 2))
        assert call(T, H, token, head) == (2 if overlap else 3), (T, H, token, head)
        seen.add(overlap)
    assert seen == {True, False}
    # the far ends of the accepted range
    assert call(2 ** 31 - 1, 65535, 8 * 16, 8) == 2 and call(2 ** 20, 65535, 65535 * 8, 8) == 3
    assert call(2 ** 20, 65535, 8, 2 ** 23) == 3 and call(2 ** 20, 65535, 8, 2 ** 23 - 8) == 2


def test_steps_of_one_batch_do_not_share_their_size():
    batch = q.KVBatch.__new__(q.KVBatch)                       # (its constructor wants tensors on a GPU)
    batch.desc = q.KVBatchDesc(FAKE, FAKE, FAKE, 2, 4, 3, 0, 0)

    def read(r):
        d = ctypes.cast(r, ctypes.POINTER(q.KVBatchDesc)).contents
        return d.T, d.max_tok, d.B

    five, nine = batch.ref(5), batch.ref(9)
    assert read(five) == (5, 3, 2) and read(nine) == (9, 3, 2)
    batch.desc.max_tok = 7                                     # what is written into the batch's own descriptor counts
    assert read(batch.ref(9)) == (9, 7, 2) and read(nine) == (9, 3, 2)
    refs = [batch.ref(t) for t in range(1, 300)]               # (the ones kept are few, but all stay good)
    assert [read(r) for r in refs] == [(t, 7, 2) for t in range(1, 300)]
    assert batch.ref(299) is refs[-1] and len(batch.desc.refs) <= 64


class Recorder:
    """Stands for the library: keeps the arguments of a call, as the 32-bit ones arrive."""
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        types = q.SIGNATURES[name][1]
        return lambda *args: self.calls.append([t(x).value if t is ctypes.c_int32 else x for t, x in zip(types, args)]) or 0


def test_numbers_beyond_32_bits_are_not_cut_down(monkeypatch):
    i32 = torch.int32
    monkeypatch.setattr(q, "_ptr", lambda t: FAKE)
    monkeypatch.setattr(q, "_rows", lambda t, heads, dim, name: (FAKE, heads * dim))
    lib = Recorder()
    monkeypatch.setattr(q, "load", lambda: lib)
    tables = torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32), torch.zeros(1, 4, dtype=i32)
    with pytest.raises(ValueError, match="max_tok does not fit"):
        q.KVBatch(*tables, 2 ** 32 + 3)
    with pytest.raises(ValueError, match="rot does not fit"):
        q.qspec_rotary_turns(2 ** 32 + 64)
    u = torch.zeros(1, 1, 16, 64, dtype=torch.uint8)
    cache = q.KVCache(u, u, torch.zeros(1, 1, dtype=torch.int8), torch.zeros(1, 1, dtype=torch.int8))
    x, ws = torch.zeros(2, 1, 64, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.uint8)
    for window, arrives in ((0, 0), (5, 5), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1), (-1, -1)):
        q.qspec_kv_attention(cache, q.KVBatch(*tables, 2), x, x, ws, window=window, stream=0)
        assert lib.calls[-1][6] == arrives                      # (a window beyond every position hides none)
    with pytest.raises(ValueError, match="window does not fit"):
        q.qspec_kv_attention(cache, q.KVBatch(*tables, 2), x, x, ws, window=-2 ** 32, stream=0)


def test_attention_refuses_scales_that_leave_fp32_in_powers_of_two(lib):
    """Scores are taken in powers of two: scale * log2(e) has to be finite.  (A misaligned q is looked at afterwards.)"""
    W = lib.qspec_kv_attention_workspace_size()
    cache = ctypes.byref(q.KVCacheDesc(FAKE, FAKE, FAKE, FAKE, 10, 8, 64, 128, 0))
    batch = ctypes.byref(q.KVBatchDesc(FAKE, FAKE, FAKE, 2, 4, 3, 0, 6))
    for scale, code in ((2.0 ** 127, 3), (-2.0 ** 127, 3), (0.0, 3), (3e38, 1), (-3e38, 1)):
        assert lib.qspec_kv_attention(cache, batch, FAKE + 2, 4096, 32, scale, 0, None, FAKE, 4096, None, FAKE, W, None) == code, scale
