"""What the beam search of the attention model refuses (CPU: it is refused before the model is asked for anything)."""
import types

import pytest
import torch

from quantized_speculative_decoding_qspec_gb300 import attention_lm as lm


def model(pages=64, page=16):
    cache = types.SimpleNamespace(page=page, k=torch.zeros(pages, 1))
    return types.SimpleNamespace(cache=cache, V=100, device="cpu")


@pytest.mark.parametrize("prompts,more,match", [
    ([], {}, "at least one"), ([[1]], {"beams": 0}, "at least one"), ([[1]], {"max_new": 0}, "at least one"), ([[]], {}, "1 to 256 tokens"),
    ([[1] * 9], {"max_len": 8}, "1 to 8 tokens"), ([[1]], {"end_tok": 100}, "end_tok"), ([[1]], {"end_tok": -1}, "end_tok"),
    ([[1]] * 2, {"beams": 8, "max_new": 17}, "too few pages")])
def test_refusals(prompts, more, match):
    with pytest.raises(ValueError, match=match):
        lm.Beams(model(), prompts, **more)
