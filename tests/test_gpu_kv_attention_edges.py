"""qspec_kv_attention at the edges of what it accepts, against the definition in 64 bits (kv_ref.attention and its tolerances)."""
import pytest
import torch

import kv_ref as ref
from gpu_util import DEV, lib
from test_gpu_kv_attention import check, queries, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [0, 1, 25, 2 ** 31 - 1])
@pytest.mark.parametrize("tok,kv,heads_q", [(40, 30, 1), (40, 30, 4), (40, 1, 2), (64, 40, 1)])
def test_more_new_tokens_than_positions(tok, kv, heads_q, window):
    """The first tokens lie before the cache and see nothing; the others see what a window of any size leaves."""
    q = lib()
    bt = ref.Batch(101, [tok], [tok], 1, 16, 64)
    bt.kv = [kv]
    qq = queries(31, tok, heads_q, 64)
    out, lse = run(q, bt, qq, window=window)
    q.qspec_check_status()
    check((out, lse), bt, qq, window=window)
    assert bool((out[:tok - kv] == 0).all()) and bool((lse[:tok - kv] == float("-inf")).all())


@pytest.mark.parametrize("B,heads_q,heads,dim", [(129, 4, 2, 64), (240, 2, 1, 128), (375, 2, 2, 128), (1024, 1, 1, 128), (1024, 1, 1, 64),
                                                 (256, 20, 1, 128), (150, 66, 1, 128), (520, 65, 1, 64)])
def test_many_sequences(B, heads_q, heads, dim):
    """Single tokens of up to 1024 sequences (a thread of the share-out then takes several), some with nothing cached."""
    q = lib()
    g = torch.Generator().manual_seed(B)
    kv = torch.randint(1, 40, (B,), generator=g).tolist()
    kv[B // 2], kv[B - 1] = 300, 70
    tok = [int(x) for x in torch.rand(B, generator=g) < 0.9]
    tok[B // 2] = tok[B - 1] = 1
    bt = ref.Batch(111, tok, kv, heads, 16, dim)
    qq = queries(33, bt.T, heads_q, dim)
    check(run(q, bt, qq), bt, qq)
    q.qspec_check_status()
