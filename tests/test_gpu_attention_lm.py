"""The attention model's serving loop: what it emits are the W4A16 model's greedy choices, whatever was drafted,
and the cache holds what one pass over the finished sequences writes."""
import pytest
import torch

import kv_ref as ref
from gpu_util import DEV, lib
from quantized_speculative_decoding_qspec_gb300 import attention_lm as lm

pytestmark = pytest.mark.gpu


def words(V, banned):
    w = torch.full(((V + 31) // 32,), -1, dtype=torch.int64)
    for t in banned:
        w[t // 32] &= ~(1 << (t % 32))
    return (w & 0xFFFFFFFF).where((w & 0xFFFFFFFF) < 2 ** 31, (w & 0xFFFFFFFF) - 2 ** 32).to(torch.int32).to(DEV)


@pytest.mark.parametrize("gamma,page,penalties,banned", [(3, 16, None, ()), (4, 64, (1.2, 0.3, 0.1), range(0, 512, 3)), (1, 32, (1.1, 0.0, 0.5), ())])
def test_emitted_tokens_are_the_target_models_choices(gamma, page, penalties, banned):
    q = lib()
    V = 512
    model = lm.AttentionLM(V=V, width=256, heads_q=4, heads=2, dim=64, page=page, n_pages=96, seed=3)
    g = torch.Generator().manual_seed(4)
    prompts = [torch.randint(0, V, (n,), generator=g).tolist() for n in (5, 1, 40)]
    server = lm.Server(model, prompts, gamma=gamma, max_len=110, penalties=penalties, allowed=words(V, banned) if banned else None)
    for _ in range(12):
        server.step()
    q.qspec_check_status(server.vws)
    assert torch.equal(server.kv_len + 1, server.hist_len)
    cache = model.cache
    model.cache = q.new_kv_cache(96, 2, page, 64)      # a second cache, filled by one pass over each finished sequence
    for b, p in enumerate(prompts):
        n = int(server.hist_len[b])
        seq = server.hist[b:b + 1, :n - 1].contiguous()
        kv = torch.tensor([n - 1], dtype=torch.int32, device=DEV)
        batch = q.KVBatch(torch.tensor([0, n - 1], dtype=torch.int32, device=DEV), kv, server.pages[b:b + 1].contiguous(), n - 1)
        logits = model.forward(seq.view(-1), batch, draft_mode=False).double().cpu()
        h = server.hist[b, :n].cpu()
        for i in range(len(p), n):                     # token i was chosen from the logits behind token i - 1
            z, _ = ref.logits(logits[i - 1].view(1, 1, V), hist=h[None, :i], hist_len=[i], prompt_len=[len(p)],
                              pen=None if penalties is None else [penalties])
            z = z.view(V)
            for t in banned:
                z[t] = -float("inf")
            # the two passes round alike but for the order of sums and, in pages that grew, the codes: a few percent of
            # the logits' spread
            assert float(z[h[i]]) >= float(z.max()) - 0.1 * float(logits[i - 1].std()), (b, i)
        # the cached values: same keys up to the roundings of the linears and of codes under another scale
        ids = server.pages[b, :-(-(n - 1) // page)].long()
        for side in "kv":
            one = cache.values(side)[ids].permute(1, 0, 2, 3).reshape(2, -1, 64)[:, :n - 1]
            two = model.cache.values(side)[ids].permute(1, 0, 2, 3).reshape(2, -1, 64)[:, :n - 1]
            assert float((one - two).norm()) <= 2 * ref.E4M3 * float(two.norm())
    q.qspec_check_status()
