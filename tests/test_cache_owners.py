"""A cache's pages are shared out by one serving loop or beam search at a time: whoever had it before is refused (no GPU)."""
import types

import pytest
import torch

from quantized_speculative_decoding_qspec_gb300 import attention_lm as lm


@pytest.fixture
def model(monkeypatch):
    calls = []
    fake = types.SimpleNamespace(
        new_beam_workspace=lambda *a, **k: None, new_verify_workspace=lambda *a, **k: None, KVPrefixes=lambda *a: None,
        KVBatch=lambda *a: None, qspec_kv_pages=lambda *a, **k: calls.append("pages"), qspec_kv_copy_pages=lambda *a, **k: calls.append("copies"))
    monkeypatch.setattr(lm, "q", fake)
    for cls in (lm.Server, lm.Beams):
        monkeypatch.setattr(cls, "_prefill", lambda self, prompts: None)

    def forward(*a, **k):
        raise Reached
    return types.SimpleNamespace(cache=types.SimpleNamespace(page=16, k=torch.zeros(64, 1)), V=100, device="cpu", forward=forward, calls=calls)


class Reached(Exception):
    pass


MAKE = {"server": lambda m: lm.Server(m, [[1, 2]], gamma=1, max_len=20), "beams": lambda m: lm.Beams(m, [[1, 2]], beams=2, max_len=20, max_new=5)}


@pytest.mark.parametrize("first", MAKE)
@pytest.mark.parametrize("second", MAKE)
def test_the_one_before_is_refused(model, first, second):
    one = MAKE[first](model)
    with pytest.raises(Reached):
        one.step()
    two = MAKE[second](model)
    with pytest.raises(ValueError, match="cache"):
        one.step()
    with pytest.raises(Reached):
        two.step()


def test_a_cache_of_its_own_stays(model):
    one = MAKE["server"](model)
    other = types.SimpleNamespace(**{**vars(model), "cache": types.SimpleNamespace(page=16, k=torch.zeros(64, 1))})
    MAKE["beams"](other)
    with pytest.raises(Reached):
        one.step()


def test_what_is_refused_takes_no_cache(model):
    one = MAKE["beams"](model)
    with pytest.raises(ValueError, match="too few pages"):
        lm.Server(model, [[1]] * 100, gamma=1, max_len=20)
    with pytest.raises(ValueError, match="too few pages"):
        lm.Beams(model, [[1]] * 100, beams=2)
    def refuses(*a, **k):
        raise ValueError("invalid beam shape")
    lm.q.new_beam_workspace = lm.q.new_verify_workspace = refuses
    for make in MAKE.values():
        with pytest.raises(ValueError, match="invalid beam shape"):
            make(model)
    with pytest.raises(Reached):
        one.step()


def test_closed_beams_take_no_step_and_give_their_pages_back_once(model):
    search = MAKE["beams"](model)
    model.calls.clear()
    search.close()
    assert model.calls == ["pages"]
    search.close()
    assert model.calls == ["pages"]
    with pytest.raises(ValueError, match="closed"):
        search.step()
