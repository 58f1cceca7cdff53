"""qspec_logits_adjust on the longest histories that a call accepts: 2^31 - 1 tokens of a sequence."""
import pytest
import torch

from gpu_util import DEV, lib

pytestmark = pytest.mark.gpu

N = 2 ** 31 - 1


def long_history():
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("not enough free memory")
    return torch.empty(1, N, dtype=torch.int32, device=DEV)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_the_last_tokens_of_the_longest_history_count():
    """The last 5000 tokens are generated ones, the rest the prompt; a step of the counting loop ends beyond 2^31."""
    q = lib()
    V, made = 2056, 5000
    hist = long_history()
    hist.random_(0, V // 2)                                 # ids of the upper half never occur in the prompt
    g = torch.Generator().manual_seed(1)
    tail = torch.randint(0, V, (made,), generator=g, dtype=torch.int32)
    hist[0, N - made:] = tail.to(DEV)
    x = (4 * torch.randn(1, 1, V, generator=g)).to(torch.bfloat16)
    rep, freq, pres = 1.25, 0.125, 0.5
    out = torch.empty_like(x, device=DEV)
    q.qspec_logits_adjust(x.to(DEV), out, hist=hist, hist_len=i32([N]), prompt_len=i32([N - made]),
                          penalties=torch.tensor([[rep, freq, pres]], device=DEV))
    q.qspec_check_status()
    c = torch.bincount(tail.long(), minlength=V).double()
    seen = (torch.arange(V) < V // 2) | (c > 0)
    z = x.view(V).double()
    z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z) - freq * c - pres * (c > 0)
    # half a bf16 step, and five fp32 roundings of values below 64
    assert bool(((out.view(V).double().cpu() - z).abs() <= 2.0 ** -8 * z.abs() + 5 * 64 * 2.0 ** -24).all())


@pytest.mark.parametrize("V", [16, 9])
def test_a_draft_token_on_top_of_the_largest_count(V):
    q = lib()
    hist = long_history().fill_(7)
    x = torch.full((1, 2, V), 3.0, dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(x)
    q.qspec_logits_adjust(x, out, draft_tok=i32([[7]]), hist=hist, hist_len=i32([N]),
                          penalties=torch.tensor([[1.0, 2.0 ** -31, 0.0]], device=DEV))
    q.qspec_check_status()
    want = torch.full((2, V), 3.0)
    want[:, 7] = 2.0                                        # (2^31 - 1) / 2^31 and 1: the same in bf16
    assert torch.equal(out[0].float().cpu(), want)
