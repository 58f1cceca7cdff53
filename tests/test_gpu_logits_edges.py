"""qspec_logits_adjust at the ends of fp32's range."""
import pytest
import torch

from gpu_util import DEV, lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [64, 65])
@pytest.mark.parametrize("rep", [2.0 ** -149, 3e-39, 2.0 ** -127, 2.0 ** -126, 1e-30, 1e30, 2.0 ** 126, 2.0 ** 127, 3e38])
def test_repetition_penalties_of_any_size(V, rep):
    """Quotients and products as far as fp32 holds them: half a bf16 step, and three fp32 roundings."""
    q = lib()
    rep = float(torch.tensor(rep, dtype=torch.float32))
    e = torch.linspace(-130, 127, V, dtype=torch.float64)
    x = (torch.where(torch.arange(V) % 2 == 0, 1.0, -1.0) * torch.exp2(e)).to(torch.bfloat16)
    out = torch.empty(1, 1, V, dtype=torch.bfloat16, device=DEV)
    hist = torch.arange(V, dtype=torch.int32, device=DEV)[None]
    q.qspec_logits_adjust(x.view(1, 1, V).to(DEV), out, hist=hist, hist_len=torch.tensor([V], dtype=torch.int32, device=DEV),
                          penalties=torch.tensor([[rep, 0.0, 0.0]], device=DEV))
    q.qspec_check_status()
    z = x.double()
    want = torch.where(z > 0, z / rep, z * rep)
    got = out.view(V).double().cpu()
    normal = (want.abs() >= 2.0 ** -126) & (want.abs() < 2.0 ** 127)    # (beyond: infinity or fewer bits)
    assert int(normal.sum()) >= 4
    err = (got - want).abs()
    assert bool((err <= (2.0 ** -8 + 3 * 2.0 ** -24) * want.abs())[normal].all())
    small = want.abs() < 2.0 ** -126
    assert bool((err <= 2.0 ** -133)[small].all())
    assert bool((got.sign() == want.sign())[normal].all()) and not bool(torch.isnan(got).any())
