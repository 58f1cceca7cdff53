"""Beams that nothing continues (a prompt whose logits are NaN: the selection gives parent -1) hold no pages and no positions, so that the
next step writes nowhere on their account; a beam's length is its parent's (no GPU: what the page tables are asked for)."""
import types

import pytest
import torch

from quantized_speculative_decoding_qspec_gb300 import attention_lm as lm


def gather(src, idx, out):
    out.copy_(torch.where(idx[:, None] >= 0, src[idx.long().clamp(min=0)], torch.zeros_like(src[:1])))


@pytest.fixture
def search(monkeypatch):
    asked = []

    def pages(table, room, keep, need, refs, page, new, *rest, parent=None):
        asked.append({"room": room.tolist(), "keep": keep.tolist(), "need": need.tolist(), "parent": parent.tolist()})
    monkeypatch.setattr(lm, "q", types.SimpleNamespace(
        new_beam_workspace=lambda *a, **k: None, KVPrefixes=lambda *a: None, KVBatch=lambda *a: None, qspec_kv_pages=pages,
        qspec_kv_copy_pages=lambda *a, **k: None, qspec_gather_rows=gather))
    monkeypatch.setattr(lm.Beams, "_prefill", lambda self, prompts: None)
    model = types.SimpleNamespace(cache=types.SimpleNamespace(page=16, k=torch.zeros(64, 1)), V=100, device="cpu")
    s = lm.Beams(model, [[1] * 20, [2] * 7], beams=2, max_len=20, max_new=5, end_tok=99)
    s.asked = asked
    return s


def chosen(s, parent, tok):
    s.parent, s.tok = torch.tensor(parent, dtype=torch.int32).view(2, 2), torch.tensor(tok, dtype=torch.int32).view(2, 2)


def test_a_prompt_without_candidates(search):
    chosen(search, [0, 0, -1, -1], [5, 6, -1, -1])           # (rows of the prompts)
    search._fork(search.prompt_len)
    assert search.asked[-1] == {"room": [20, 7], "keep": [20, 20, 0, 0], "need": [21, 21, 0, 0], "parent": [0, 0, -1, -1]}
    assert search.length.tolist() == [21, 21, 0, 0]
    assert search.tokens[:, :, 0].tolist() == [[5, 6], [-1, -1]]


def test_a_beam_that_is_lost_and_taken_up_again(search):
    chosen(search, [0, 0, 1, -1], [5, 6, 7, -1])
    search._fork(search.prompt_len)
    assert search.length.tolist() == [21, 21, 8, 0]
    chosen(search, [1, 0, 2, 2], [8, 99, 9, 10])             # both from the one that is left
    search._fork(search.length)
    assert search.asked[-1] == {"room": [21, 21, 8, 0], "keep": [21, 21, 8, 8], "need": [22, 22, 9, 9], "parent": [1, 0, 2, 2]}
    assert search.length.tolist() == [22, 22, 9, 9]
    assert search.tokens[:, :, :2].tolist() == [[[6, 8], [5, 99]], [[7, 9], [7, 10]]]
    assert search.done.tolist() == [[0, 1], [0, 0]] and search.added.tolist() == [[2, 2], [2, 2]]
    chosen(search, [1, 0, -1, -1], [99, 3, -1, -1])
    search._fork(search.length)
    assert search.length.tolist() == [23, 23, 0, 0]
    assert search.tokens[0, :, :3].tolist() == [[5, 99, -1], [6, 8, 3]]
    assert (search.tokens[1] == -1).all()
