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
