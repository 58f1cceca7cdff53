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


@pytest.mark.parametrize("heads_q", [2, 20, 70])               # both decode kernels, the prefill kernel
@pytest.mark.parametrize("magnitude", [20, 21, 22, 23, 24, 25, 26, 27, 28, 29, 31])
def test_scores_so_large_that_their_steps_are_coarse(magnitude, heads_q):
    """A score of about 2^magnitude powers of two, and one 12 to 20 powers of two above it a few tiles later: all
    values are 1, so the output is 1 whatever the weights round to.  (700 sequences of seven kinds: a CTA walks several tiles.)"""
    q = lib()
    P, D, N, B = 128, 64, 300, 700
    scale = next(s for k in range(-4, 5) for s in [torch.tensor(0.6931472, dtype=torch.float32).view(torch.int32).add(k).view(torch.float32)]
                 if float(s * torch.tensor(1.44269504088896, dtype=torch.float32)) == 1.0)
    above = torch.tensor([12, 13, 14, 15, 16, 18, 20], dtype=torch.float64)
    kinds, n = len(above), -(-N // P)
    k, v = torch.zeros(kinds * n, 1, P, D, dtype=torch.uint8), torch.full((kinds * n, 1, P, D), 0x38, dtype=torch.uint8)
    for b in range(kinds):
        k[b * n, 0, 0, 0] = k[b * n + 1, 0, 0, 0] = 0x78                    # 2^8
        k[b * n + 1, 0, 0, 1] = ref.e4m3(above[b:b + 1])[0]
    exps = torch.zeros(kinds * n, 1, dtype=torch.int8)
    table = torch.arange(kinds * n, dtype=torch.int32, device=DEV).view(kinds, n).repeat(B // kinds, 1)
    cache = q.KVCache(k.to(DEV), v.to(DEV), exps.to(DEV), exps.clone().to(DEV))
    batch = q.KVBatch(torch.arange(B + 1, dtype=torch.int32, device=DEV), torch.full((B,), N, dtype=torch.int32, device=DEV),
                      table, 1)
    qq = torch.zeros(B, heads_q, D, dtype=torch.bfloat16, device=DEV)
    qq[..., 0], qq[..., 1] = 2.0 ** (magnitude - 8), 1.0
    out, lse = torch.empty_like(qq), torch.empty(B, heads_q, device=DEV)
    q.qspec_kv_attention(cache, batch, qq, out, q.new_kv_attention_workspace(), scale=float(scale), lse=lse)
    q.qspec_check_status()
    # the weights' rounding to fp16 (2^-11), the output's to bf16
    assert float((out.double() - 1).abs().max()) <= 2.0 ** -8 + 2.0 ** -10
    # the score's own rounding (half a step of fp32 and of its product), and the logarithm of at most two such weights
    want = (2.0 ** magnitude + above.to(DEV).repeat(B // kinds)[:, None]) * 0.6931471805599453
    assert float((lse.double() - want).abs().max()) <= 2.0 ** (magnitude - 22) + 1


@pytest.mark.parametrize("tok,kv,heads_q,heads,dim", [([140], [300], 2, 1, 128), ([200, 70], [512, 129], 4, 2, 128), ([64, 1], [1000, 77], 8, 1, 128)])
def test_prompt_chunks_over_long_pages(tok, kv, heads_q, heads, dim):
    """More than 64 rows a key head, heads of 128, pages of 128 slots."""
    q = lib()
    bt = ref.Batch(121, tok, kv, heads, 128, dim)
    qq = queries(35, bt.T, heads_q, dim)
    check(run(q, bt, qq), bt, qq)
    q.qspec_check_status()


@pytest.mark.parametrize("heads_q", [2, 20, 70])               # both decode kernels, the prefill kernel
@pytest.mark.parametrize("page,dim", [(16, 64), (64, 128), (128, 64)])
def test_the_tokens_of_bad_pages_are_left_out(page, dim, heads_q, monkeypatch):
    """The first, a middle and the last page of a sequence are missing: the others' tokens alone count."""
    q = lib()
    tok, kv = [1, 2], [90, 5 * page - 7]
    bt = ref.Batch(131, tok, kv, 1, page, dim)
    qq = queries(37, bt.T, heads_q, dim)
    cache, batch = bt.gpu(q)
    missing = (0, 2, 4)
    batch.pages[1, 0], batch.pages[1, 2], batch.pages[1, 4] = -1, bt.n_pages, 2 ** 31 - 1
    qg = qq.to(DEV)
    out, lse = torch.full_like(qg, 77.0), torch.empty(qq.shape[:2], device=DEV)
    q.qspec_kv_attention(cache, batch, qg, out, q.new_kv_attention_workspace(), lse=lse)
    with pytest.raises(q.QSpecError, match="INVALID_ARG"):
        q.qspec_check_status()
    seen = ref.visible

    def visible(i, n, length, *args):
        see = seen(i, n, length, *args)
        if length == kv[1]:
            for p in missing:
                see[p * page:(p + 1) * page] = False
        return see

    monkeypatch.setattr(ref, "visible", visible)
    check((out, lse), bt, qq)
