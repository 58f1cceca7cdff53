"""Attention over shared prefixes where whole row tiles see nothing: sequences with new tokens and no positions (padding that an append
leaves out), among groups that do.  Their outputs are 0 and -inf, the others' those of the 64-bit reference."""
import numpy as np
import pytest
import torch

import kv_ref as ref
from gpu_util import lib
from test_gpu_kv_shared import call, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tok", [1, 5, 20, 130])        # 4, 20, 80 and 520 rows a sequence and key head
@pytest.mark.parametrize("members,empty", [([1], [0]), ([3], [0, 1, 2]), ([2, 4], [2, 3, 4, 5]), ([4, 2], [0, 1, 2, 3]), ([3, 3], [1])])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64)])
def test_tiles_that_see_nothing(tok, members, empty, dim, page):
    q = lib()
    B = sum(members)
    toks = [tok + b % 3 for b in range(B)]
    kv = [0 if b in empty else 200 + 37 * b for b in range(B)]
    bt = ref.Batch(tok + B, toks, kv, 2, page, dim)
    bt.members = members
    bt.table = torch.cat([bt.table, torch.full((B, 4), -7, dtype=torch.int32)], 1)     # room for a prefix of 60 in every table
    prefix = [60 if m == 1 else 0 for m in members]      # nothing in common, or all of one sequence
    qt, out, lse = call(q, bt, 8, prefix)
    q.qspec_check_status()
    check(bt, qt, out, lse)
    cu = np.cumsum([0] + toks)
    for b in empty:
        assert bool((out[cu[b]:cu[b + 1]] == 0).all()) and bool(torch.isneginf(lse[cu[b]:cu[b + 1]]).all())


@pytest.mark.parametrize("tok", [2, 30])
def test_a_group_that_sees_nothing_beside_a_shared_prefix(tok):
    """The prefix of the empty group shrinks to nothing, whatever its length says."""
    q = lib()
    toks, kv = [tok] * 4, [150 + tok, 0, 150 + tok, 0]
    bt = ref.Batch(3, toks, kv, 1, 32, 64)
    bt.members = [1, 1, 1, 1]
    qt, out, lse = call(q, bt, 4, [100, 100, 150, 0], window=0)
    q.qspec_check_status()
    check(bt, qt, out, lse)
