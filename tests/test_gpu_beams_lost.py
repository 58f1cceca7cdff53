"""A prompt whose logits are NaN loses its beams; the other prompts' beams go on as if it were not there, page for page."""
import math

import pytest
import torch

from gpu_util import lib
from quantized_speculative_decoding_qspec_gb300 import attention_lm as lm
from test_gpu_attention_lm_beams import one_pass

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page,beams", [(16, 4), (64, 3)])
def test_the_other_prompts_go_on(page, beams):
    q = lib()
    V, new = 512, 18
    model = lm.AttentionLM(V=V, width=256, heads_q=4, heads=2, dim=64, page=page, n_pages=160, seed=5)
    model.E[V - 1] = math.nan
    g = torch.Generator().manual_seed(6)
    prompts = [torch.randint(0, V - 1, (n,), generator=g).tolist() for n in (70, 5, page)]
    prompts[1][-1] = V - 1                         # (an earlier one leaves zeros in the cache, and finite logits)
    search = lm.Beams(model, prompts, beams=beams, max_len=80, max_new=new, end_tok=7)
    for _ in range(new - 1):
        search.step()
    with pytest.raises(q.QSpecError, match="QSPEC_ERR_INVALID_ARG"):
        q.qspec_check_status()
    refs, table, length = search.refs.cpu().tolist(), search.tables[0].cpu().tolist(), search.length.cpu().tolist()
    assert length[beams:2 * beams] == [0] * beams
    want = [0] * len(refs)
    for row, n in zip(table, length):
        for p in row[:-(-n // page)]:
            want[p] += 1
    assert refs == want and int(search.left) == want.count(0)
    tokens, scores = search.tokens.cpu(), search.score.cpu()
    assert bool((tokens[1] == -1).all()) and bool(torch.isneginf(scores[1]).all())
    for b in (0, 2):
        rows = [tuple(t for t in tokens[b, k].tolist() if t >= 0) for k in range(beams)]
        assert len(set(rows)) == beams
        for k, row in enumerate(rows):
            logp, std = one_pass(model, q, list(prompts[b]) + list(row))
            total = sum(float(logp[len(prompts[b]) - 1 + i, t]) for i, t in enumerate(row))
            # as for prompts that are all finite: a few percent of the logits' spread for each token
            assert abs(float(scores[b, k]) - total) <= 0.05 * std * len(row), (b, k)
    search.close()
    assert int(search.refs.abs().sum()) == 0
    q.qspec_check_status()
