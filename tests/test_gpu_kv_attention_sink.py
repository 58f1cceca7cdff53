"""qspec_kv_attention where one dominant key stands in front of a million small ones.

The cache has two pages; the tables name the second one again and again, so that long sequences cost no memory."""
import math

import pytest
import torch

from gpu_util import DEV, lib

pytestmark = pytest.mark.gpu

ONE = 0x38                                                   # 1.0 as an e4m3 code


@pytest.mark.parametrize("below", [25.5, 28.0])
@pytest.mark.parametrize("B,Hq", [(700, 1), (700, 20), (160, 128)])   # both decode kernels, the prefill kernel
def test_small_weights_behind_a_dominant_key_count(B, Hq, below):
    """The first key weighs 1 and its value is 0; the others weigh 2^-below each, and their values are 1.  There are more
    sequences than CTAs, so a CTA sees most of a sequence."""
    q = lib()
    P, D, N = 128, 64, 1 << 20
    k, v = (torch.zeros(2, 1, P, D, dtype=torch.uint8) for _ in range(2))
    k[0, 0, 0, 0] = ONE
    v[:] = ONE
    v[0, 0, 0] = 0
    exps = torch.zeros(2, 1, dtype=torch.int8)
    cache = q.KVCache(k.to(DEV), v.to(DEV), exps.to(DEV), exps.clone().to(DEV))
    table = torch.ones(B, N // P, dtype=torch.int32, device=DEV)
    table[:, 0] = 0
    batch = q.KVBatch(torch.arange(B + 1, dtype=torch.int32, device=DEV), torch.full((B,), N, dtype=torch.int32, device=DEV), table, 1)
    qq = torch.zeros(B, Hq, D, dtype=torch.bfloat16, device=DEV)
    qq[:, :, 0] = 1
    out, lse = torch.empty_like(qq), torch.empty(B, Hq, device=DEV)
    scale = float(torch.tensor(below * math.log(2), dtype=torch.float32))
    q.qspec_kv_attention(cache, batch, qq, out, q.new_kv_attention_workspace(), scale=scale, lse=lse)
    q.qspec_check_status()
    tail = (N - 1) * math.exp(-scale)
    want = tail / (1 + tail)
    # the output's rounding to bf16; the weights' rounding to fp16, half a step of 2^-24 where the largest is 2^8; a sum of
    # at most 2^14 steps in fp32 (16 keys of every 64, or 64 at a time); exponents of up to 2^5 in fp32
    tol = want * (2.0 ** -8 + 2.0 ** (below - 33) + 2.0 ** (14 - 24) + 2.0 ** (5 - 22))
    assert float((out.double() - want).abs().max()) <= tol, (float(out.min()), float(out.max()), want)
    tol_l = 2.0 ** (14 - 24) + 2.0 ** (5 - 22)
    assert float((lse.double() - (scale + math.log1p(tail))).abs().max()) <= tol_l
