"""qspec_kv_attention against the definition in 64 bits, with the tolerance that kv_ref.attention derives."""
import pytest
import torch

import kv_ref as ref
from gpu_util import DEV, lib

pytestmark = pytest.mark.gpu


def queries(seed, T, Hq, D, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (size * torch.randn(T, Hq, D, generator=g)).to(torch.bfloat16)


def run(q, bt, qq, scale=None, window=0, tree=None, ws=None, with_lse=True):
    cache, batch = bt.gpu(q)
    qg = qq.to(DEV)
    out = torch.full_like(qg, 77.0)
    lse = torch.full(qq.shape[:2], 77.0, device=DEV) if with_lse else None
    ws = q.new_kv_attention_workspace() if ws is None else ws
    q.qspec_kv_attention(cache, batch, qg, out, ws, scale=scale, window=window, lse=lse,
                         tree=tree.to(DEV) if tree is not None else None)
    return out, lse


def check(got, bt, qq, scale=None, window=0, tree=None):
    out, lse = got
    want, want_l, tol, tol_l = ref.attention(bt, qq, bt.D ** -0.5 if scale is None else scale, window, tree)
    err = (out.double().cpu() - want).abs()
    assert bool((err <= tol).all()), (float(err.max()), float((err - tol).max()))
    if lse is not None:
        empty = torch.isinf(want_l)
        l = lse.double().cpu()
        assert torch.equal(l[empty], want_l[empty])
        assert bool(((l - want_l).abs() <= tol_l)[~empty].all()), float((l - want_l).abs()[~empty].max())


CASES = [  # tok, kv, heads_q, heads, page, dim
    ([1], [1], 1, 1, 16, 64), ([1], [2], 4, 1, 16, 128), ([1], [517], 8, 2, 64, 128), ([1, 1, 1], [63, 64, 65], 4, 2, 64, 128),
    ([4, 4], [4, 70], 8, 2, 64, 128), ([1, 5, 2, 4], [129, 5, 16, 255], 3, 3, 16, 64), ([7, 1], [300, 1000], 14, 2, 32, 128),
    ([4], [2049], 8, 1, 128, 64), ([3, 3], [200, 131], 16, 2, 128, 128), ([33], [33], 2, 1, 16, 64), ([70, 3], [100, 3], 8, 1, 32, 128),
    ([150], [403], 4, 1, 64, 128), ([257], [257], 2, 2, 64, 64), ([140, 2, 129], [141, 300, 129], 8, 2, 128, 64), ([260], [1300], 3, 1, 64, 128),
    ([1], [700], 128, 1, 64, 128), ([2, 0, 1], [40, 33, 0], 2, 2, 16, 64)]


@pytest.mark.parametrize("tok,kv,Hq,H,P,D", CASES)
def test_attention(tok, kv, Hq, H, P, D):
    q = lib()
    if tok[-1] > kv[-1]:
        tok = tok[:-1] + [0]
    bt = ref.Batch(31 + sum(kv), tok, kv, H, P, D)
    qq = queries(5, bt.T, Hq, D)
    check(run(q, bt, qq), bt, qq)
    q.qspec_check_status()


@pytest.mark.parametrize("seed", range(6))
def test_items_cut_into_many_parts(seed):
    """Sequences whose tiles are spread over more CTAs than meet at once, at lengths that move the cuts about; the
    same numbers again from the same workspace."""
    q = lib()
    g = torch.Generator().manual_seed(100 + seed)
    B = 4 + 2 * seed
    kv = torch.randint(900, 1500, (B,), generator=g).tolist()
    bt = ref.Batch(200 + seed, [2] * B, kv, 8, 64, 64)
    qq = queries(20 + seed, bt.T, 8, 64)
    ws = q.new_kv_attention_workspace()
    a = run(q, bt, qq, ws=ws)
    check(a, bt, qq)
    for _ in range(3):
        b = run(q, bt, qq, ws=ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 129, 100000])
@pytest.mark.parametrize("tok,kv,Hq,H,P,D", [([4, 1], [200, 333], 4, 2, 16, 64), ([140], [300], 4, 1, 64, 128)])
def test_window(tok, kv, Hq, H, P, D, window):
    q = lib()
    bt = ref.Batch(41, tok, kv, H, P, D)
    qq = queries(6, bt.T, Hq, D)
    check(run(q, bt, qq, window=window), bt, qq, window=window)


def trees(seed, tok):
    g = torch.Generator().manual_seed(seed)
    words = []
    for n in tok:
        own = []
        for j in range(n):
            p = int(torch.randint(-1, j, (1,), generator=g)) if j else -1
            own.append((own[p] if p >= 0 else 0) | 1 << j)
        words += own
    return torch.tensor([w - 2 ** 64 if w >= 2 ** 63 else w for w in words], dtype=torch.int64)


@pytest.mark.parametrize("tok,kv,Hq,H,P,D", [([7], [7], 2, 2, 16, 64), ([5, 31, 1], [77, 31, 64], 4, 2, 16, 64), ([64, 64], [64, 200], 2, 1, 64, 128),
                                             ([31, 20], [150, 129], 8, 1, 32, 128)])
def test_tree(tok, kv, Hq, H, P, D):
    q = lib()
    bt = ref.Batch(51, tok, kv, H, P, D)
    qq = queries(7, bt.T, Hq, D)
    tree = trees(8, tok)
    check(run(q, bt, qq, tree=tree), bt, qq, tree=tree)
    # a chain's tree words are the causal mask
    chain = torch.tensor([(1 << (i + 1)) - 1 if i < 62 else ((1 << (i + 1)) - 1) - (2 ** 64 if i == 63 else 0) for n in tok for i in range(n)],
                         dtype=torch.int64)
    a, b = run(q, bt, qq, tree=chain), run(q, bt, qq)
    check(a, bt, qq)
    check(b, bt, qq)


def test_rows_that_see_nothing():
    """Tree words of 0 without a prefix, and bits beyond the sequence's nodes: zeros and -inf, no NaN."""
    q = lib()
    bt = ref.Batch(61, [3, 2], [3, 40], 2, 16, 64)
    tree = torch.tensor([0, 1, 1 << 40, 0, -1], dtype=torch.int64)
    qq = queries(9, 5, 4, 64)
    out, lse = run(q, bt, qq, tree=tree)
    check((out, lse), bt, qq, tree=tree)
    assert bool((out[[0, 2]] == 0).all()) and bool((lse[[0, 2]] == float("-inf")).all())
    # more new tokens than cached positions: the first ones lie before the cache
    bt = ref.Batch(62, [40], [40], 2, 16, 64)
    cache, batch = bt.gpu(q)
    batch.kv_len.fill_(30)
    qg = queries(10, 40, 4, 64).to(DEV)
    out, lse, ws = torch.empty_like(qg), torch.empty(40, 4, device=DEV), q.new_kv_attention_workspace()
    q.qspec_kv_attention(cache, batch, qg, out, ws, lse=lse)
    q.qspec_check_status()
    assert bool((out[:10] == 0).all()) and bool((lse[:10] == float("-inf")).all())
    assert bool(torch.isfinite(lse[10:]).all())


@pytest.mark.parametrize("spread", [0.0, 6.0])
@pytest.mark.parametrize("size", [1e-3, 1.0, 30.0])
def test_magnitudes(size, spread):
    """Peaked and flat softmaxes, pages whose scales differ by many powers of two."""
    q = lib()
    bt = ref.Batch(71, [3, 130], [500, 260], 2, 16, 128, spread=spread)
    qq = queries(11, bt.T, 4, 128, size)
    check(run(q, bt, qq), bt, qq)


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0])
def test_scales(scale):
    q = lib()
    bt = ref.Batch(73, [2, 70], [90, 200], 1, 32, 64, spread=0.0)
    qq = queries(12, bt.T, 4, 64)
    check(run(q, bt, qq, scale=scale), bt, qq, scale=scale)


def test_range_of_queries():
    """Queries far outside fp16's range and rows of zeros; a NaN query spoils its own row only."""
    q = lib()
    bt = ref.Batch(75, [6, 131], [80, 150], 1, 16, 64, spread=0.0)
    qq = queries(13, bt.T, 4, 64, 1.0)
    qq[0] *= 2.0 ** 40
    qq[1] = 0
    qq[2] *= 2.0 ** -60
    qq[10, 1] *= 2.0 ** 30
    clean = qq.clone()
    qq[3, 2, 5] = float("nan")
    qq[20, 1, 9] = float("nan")
    out, lse = run(q, bt, qq)
    assert bool(torch.isnan(out[3, 2]).all()) and bool(torch.isnan(out[20, 1]).all())
    ok = ~torch.isnan(out).any(-1).cpu()
    assert int((~ok).sum()) == 2
    clean[3, 2], clean[20, 1] = 0, 0
    want, want_l, tol, tol_l = ref.attention(bt, clean, 64 ** -0.5)
    assert bool(((out.double().cpu() - want).abs() <= tol)[ok].all())


def test_strided_queries_and_no_lse():
    q = lib()
    bt = ref.Batch(77, [3, 140], [100, 140], 2, 16, 64)
    T, Hq, D = bt.T, 4, 64
    qq = queries(14, T, Hq, D)
    want, _ = run(q, bt, qq)
    cache, batch = bt.gpu(q)
    wide = torch.full((T, Hq * D + 64), 3.0, dtype=torch.bfloat16, device=DEV)
    src = wide[:, 32:32 + Hq * D].unflatten(1, (Hq, D))
    src.copy_(qq)
    dst = torch.full((T, Hq * D + 8), 9.0, dtype=torch.bfloat16, device=DEV)
    q.qspec_kv_attention(cache, batch, src, dst[:, :Hq * D].unflatten(1, (Hq, D)), q.new_kv_attention_workspace())
    assert torch.equal(dst[:, :Hq * D].reshape(T, Hq, D), want)
    assert bool((dst[:, Hq * D:] == 9).all())


def test_one_workspace_serves_every_shape_and_runs_repeat():
    q = lib()
    ws = q.new_kv_attention_workspace()
    shapes = [([1], [3000], 8, 1, 64, 128), ([4, 4, 4], [700, 5, 1900], 8, 2, 16, 64), ([200], [900], 4, 1, 32, 128), ([1], [3000], 8, 1, 64, 128)]
    first = None
    for tok, kv, Hq, H, P, D in shapes:
        bt = ref.Batch(81, tok, kv, H, P, D)
        qq = queries(15, bt.T, Hq, D)
        a = run(q, bt, qq, ws=ws)
        check(a, bt, qq)
        b = run(q, bt, qq, ws=ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])     # the order of the sums is fixed
        if first is None:
            first = a
    assert torch.equal(first[0], a[0])


def test_bad_pages_are_reported_and_left_out():
    q = lib()
    for tok in ([2, 2], [2, 130]):
        bt = ref.Batch(83, tok, [100, 230], 2, 16, 64)
        qq = queries(16, bt.T, 4, 64)
        good = run(q, bt, qq)
        cache, batch = bt.gpu(q)
        batch.pages[1, 3] = bt.n_pages
        batch.pages[1, 5] = -2
        out, lse, ws = torch.empty_like(good[0]), torch.empty_like(good[1]), q.new_kv_attention_workspace()
        q.qspec_kv_attention(cache, batch, qq.to(DEV), out, ws, lse=lse)
        with pytest.raises(q.QSpecError, match="INVALID_ARG"):
            q.qspec_check_status()
        q.qspec_check_status()
        assert torch.equal(out[:2], good[0][:2])               # the other sequence
        assert bool(torch.isfinite(out.float()).all()) and bool(torch.isfinite(lse).all())
        batch.kv_len[1] = 1 << 20                               # beyond the page table: the sequence is left out
        out.fill_(5.0)
        q.qspec_kv_attention(cache, batch, qq.to(DEV), out, ws, lse=lse)
        with pytest.raises(q.QSpecError, match="INVALID_ARG"):
            q.qspec_check_status()
        assert torch.equal(out[:2], good[0][:2]) and bool((out[2:] == 5).all())


def test_cache_beyond_32_bit_offsets():
    """A pool of more than 2^32 bytes a side; the sequences' pages lie at its end."""
    q = lib()
    H, P, D = 8, 64, 128
    n = (1 << 32) // (H * P * D) + 40
    if torch.cuda.mem_get_info()[0] < 3 * n * H * P * D:
        pytest.skip("not enough free memory")
    cache = q.KVCache(*(torch.empty(n, H, P, D, dtype=torch.uint8, device=DEV) for _ in range(2)),
                      *(torch.empty(n, H, dtype=torch.int8, device=DEV) for _ in range(2)))
    g = torch.Generator().manual_seed(17)
    T = 150
    k, v = (torch.randn(T, H, D, generator=g).to(torch.bfloat16) for _ in range(2))
    table = torch.tensor([[n - 1, n - 30, n - 2]], dtype=torch.int32)
    batch = q.KVBatch(torch.tensor([0, T], dtype=torch.int32, device=DEV), torch.tensor([T], dtype=torch.int32, device=DEV), table.to(DEV), T)
    q.qspec_kv_append(cache, batch, k.to(DEV), v.to(DEV))
    small = ref.Batch(1, [T], [T], H, P, D)
    for side, new in (("k", k), ("v", v)):
        ref.append(small.codes[side], small.exps[side], new, small.table, small.cu, small.kv)
    for s, c, e in (("k", cache.k, cache.k_exp), ("v", cache.v, cache.v_exp)):
        for i in range(3):
            used = min(P, T - i * P)
            assert torch.equal(c[int(table[0, i]), :, :used].cpu(), small.codes[s][int(small.table[0, i]), :, :used])
    for tok in (T, 2):
        qq = queries(18, tok, 2 * H, D)
        small.tok, small.cu, small.T = [tok], [0, tok], tok
        batch.cu_tok[1] = tok
        batch.desc.max_tok = tok
        qg = qq.to(DEV)
        out = torch.empty_like(qg)
        q.qspec_kv_attention(cache, batch, qg, out, q.new_kv_attention_workspace())
        q.qspec_check_status()
        check((out, None), small, qq)


def test_other_stream_and_graph_with_growing_lengths():
    q = lib()
    bt = ref.Batch(91, [2, 2], [150, 90], 2, 16, 64)
    qq = queries(19, 4, 4, 64)
    cache, batch = bt.gpu(q)
    qg = qq.to(DEV)
    out, ws = torch.empty_like(qg), q.new_kv_attention_workspace()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    q.qspec_kv_attention(cache, batch, qg, out, ws, stream=s)
    s.synchronize()
    check((out, None), bt, qq)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.qspec_kv_attention(cache, batch, qg, out, ws)
    for kv in ([100, 33], [150, 90], [2, 90]):
        batch.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        bt.kv = kv
        check((out, None), bt, qq)
