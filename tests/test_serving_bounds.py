"""The serving loop refuses, before anything reaches a device, what its history and pages have no room for (no GPU)."""
import pytest
import torch

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


def server(kv_len, longest, max_len=10, gamma=3):
    s = lm.Server.__new__(lm.Server)
    s.model, s.B, s.gamma, s.max_len, s.longest = NoDevice(), len(kv_len), gamma, max_len, longest
    s.kv_len = torch.tensor(kv_len, dtype=torch.int32)
    s.hist_len = s.kv_len + 1
    return s


def test_a_step_beyond_max_len_is_refused():
    s = server([4, 11], longest=14)
    with pytest.raises(ValueError, match="beyond max_len 10"):
        s.step()
    assert s.longest == 11                        # read back


def test_a_step_up_to_max_len_is_taken():
    for s in (server([4, 10], longest=10), server([4, 10], longest=17)):   # within the bound; the bound too high
        with pytest.raises(NoDevice.Used):
            s.step()
        assert s.longest == 14
