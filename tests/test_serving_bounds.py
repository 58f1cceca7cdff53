"""The serving loop refuses, before anything reaches a device, what its history and pages have no room for (no GPU)."""
import pytest

from quantized_speculative_decoding_qspec_gb300 import attention_lm as lm


class NoDevice:
    """Stands for a model: any use of it shows that a call was let through."""
    class Used(Exception):
        pass

    def __getattr__(self, name):
        raise NoDevice.Used(name)


@pytest.mark.parametrize("prompts", [[[1, 2], []], [[]], [[3] * 11, [1]]])
def test_prompts_of_no_tokens_or_too_many_are_refused(prompts):
    with pytest.raises(ValueError, match="a prompt has 1 to 10 tokens"):
        lm.Server(NoDevice(), prompts, gamma=2, max_len=10)


def test_no_prompts_and_no_drafts_are_refused():
    with pytest.raises(ValueError, match="at least one"):
        lm.Server(NoDevice(), [], gamma=2)
    with pytest.raises(ValueError, match="at least one"):
        lm.Server(NoDevice(), [[1]], gamma=0)


def test_prompts_within_bounds_are_taken():
    with pytest.raises(NoDevice.Used):
        lm.Server(NoDevice(), [[1], [2] * 10], gamma=2, max_len=10)
