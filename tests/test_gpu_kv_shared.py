"""Attention over shared prefixes against the 64-bit reference of plain attention, sequence by sequence, with its tolerance (which
counts each output's roundings; the calls compute alike)."""
import math

import numpy as np
import pytest
import torch

import kv_ref as ref
from gpu_util import DEV, i32_dev, lib

pytestmark = pytest.mark.gpu


def shared_batch(seed, members, tok, prefix, own, heads, page, dim):
    """A ref.Batch of len(members) groups: group g's members[g] sequences hold the same first prefix[g] tokens, full pages shared.
    tok(rng), own(rng): new tokens, and positions behind the prefix before them, of a sequence."""
    rng = np.random.default_rng(seed)
    toks, kv, group = [], [], []
    for g, m in enumerate(members):
        for _ in range(m):
            n = tok(rng)
            toks.append(n)
            kv.append(prefix[g] + own(rng) + n)
            group.append(g)
    bt = ref.Batch(seed, toks, kv, heads, page, dim)
    for b, g in enumerate(group):
        lead = group.index(g)
        full, rest = prefix[g] // page, prefix[g] % page
        if b != lead:
            bt.table[b, :full] = bt.table[lead, :full]
            if rest:
                src, dst = int(bt.table[lead, full]), int(bt.table[b, full])
                for side in "kv":
                    bt.codes[side][dst, :, :rest] = bt.codes[side][src, :, :rest]
                    bt.exps[side][dst] = bt.exps[side][src]
    bt.members, bt.group = list(members), group
    return bt


def call(q, bt, heads_q, prefix, seed=0, scale=None, window=0, tree=None, max_tok=None, fill=7.0, members=None, qt=None, ws=None):
    cache, batch = bt.gpu(q)
    g = torch.Generator().manual_seed(seed + 100)
    if qt is None:
        qt = (torch.randn(bt.T, heads_q, bt.D, generator=g) * 2).to(torch.bfloat16)
    out = torch.full((bt.T, heads_q, bt.D), fill, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((bt.T, heads_q), fill, device=DEV)
    members = bt.members if members is None else members
    cu = [0] + [int(x) for x in np.cumsum(members)]
    most = max(sum(bt.tok[cu[i]:cu[i + 1]]) for i in range(len(members))) if max_tok is None else max_tok
    pre = q.KVPrefixes(i32_dev(cu), i32_dev(prefix), max(most, 1))
    q.qspec_kv_attention_shared(cache, batch, pre, qt.to(DEV), out, q.new_kv_attention_workspace() if ws is None else ws, scale=scale,
                                window=window, tree=None if tree is None else tree.to(DEV), lse=lse)
    return qt, out.double().cpu(), lse.double().cpu()


def check(bt, qt, out, lse, scale=None, window=0, tree=None, rows=None):
    want, want_l, tol, tol_l = ref.attention(bt, qt, bt.D ** -0.5 if scale is None else scale, window, tree)
    rows = slice(None) if rows is None else rows
    out, lse, want, want_l, tol, tol_l = (x[rows] for x in (out, lse, want, want_l, tol, tol_l))
    none = torch.isinf(want_l)
    assert torch.equal(lse[none], want_l[none]) and bool((out[none] == 0).all())
    assert bool(((out - want).abs() <= tol).all()), float(((out - want).abs() / tol.clamp(min=1e-30)).max())
    assert bool(((lse - want_l)[~none].abs() <= tol_l[~none]).all())


SHAPES = [  # members, tokens, prefix, own positions, heads of queries and keys
    ([4], (1, 1), [200], (0, 30), 4, 1),               # 16 rows
    ([3, 1, 2], (1, 4), [300, 64, 17], (0, 90), 4, 2),
    ([5, 5], (1, 1), [129, 500], (0, 200), 8, 1),      # 40 rows
    ([2, 8], (2, 7), [70, 640], (0, 10), 2, 1),
    ([40], (1, 1), [1000], (0, 300), 8, 2),            # 160 rows: tensor cores
    ([3, 9], (1, 30), [333, 90], (0, 140), 7, 1),
    ([2], (70, 300), [260], (0, 50), 2, 1),            # row tiles of one sequence
    ([130, 2], (1, 2), [50, 900], (0, 3), 4, 2),       # more sequences than a tile has
]


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 16), (64, 128), (128, 64), (128, 32)])
def test_groups(shape, dim, page):
    q = lib()
    members, tok, prefix, own, hq, hk = SHAPES[shape]
    bt = shared_batch(shape * 7 + page, members, lambda r: int(r.integers(tok[0], tok[1] + 1)), prefix,
                      lambda r: int(r.integers(own[0], own[1] + 1)), hk, page, dim)
    qt, out, lse = call(q, bt, hq, prefix, seed=shape)
    check(bt, qt, out, lse)
    q.qspec_check_status()


@pytest.mark.parametrize("window", [1, 33, 150, 2 ** 31 - 1])
@pytest.mark.parametrize("members,tok", [([4, 2], 1), ([6], 5), ([20], 6)])
def test_windows(members, tok, window):
    q = lib()
    prefix = [200] * len(members)
    bt = shared_batch(window % 97, members, lambda r: tok, prefix, lambda r: int(r.integers(0, 100)), 2, 32, 64)
    qt, out, lse = call(q, bt, 8, prefix, window=window)
    check(bt, qt, out, lse, window=window)
    q.qspec_check_status()


def test_pages_before_a_window_are_not_read():
    q = lib()
    for members, tok in (([4], 1), ([20], 5)):
        bt = shared_batch(3, members, lambda r: tok, [200], lambda r: 80, 1, 16, 64)
        qt, out, lse = call(q, bt, 4, [200], window=40)
        bt.table[:, :14] = -9                      # positions 0 .. 223: the windows begin at 241
        _, out2, lse2 = call(q, bt, 4, [200], window=40)
        q.qspec_check_status()
        assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("members,nodes,hq,hk", [([3, 2], 7, 4, 2), ([4], 31, 4, 1), ([2, 2], 64, 2, 2)])
def test_trees(members, nodes, hq, hk):
    q = lib()
    prefix = [130] * len(members)
    bt = shared_batch(nodes, members, lambda r: int(r.integers(1, nodes + 1)), prefix, lambda r: int(r.integers(0, 40)), hk, 64, 64)
    rng = np.random.default_rng(1)
    words = []
    for n in bt.tok:
        anc = []
        for j in range(n):
            p = int(rng.integers(-1, j)) if j else -1
            anc.append((anc[p] if p >= 0 else 0) | 1 << j)
        if n > 3:
            anc[3] = 0                             # a node that sees none of the tree
        words += anc
    tree = torch.from_numpy(np.array(words, dtype=np.uint64).view(np.int64))
    qt, out, lse = call(q, bt, hq, prefix, tree=tree)
    check(bt, qt, out, lse, tree=tree)
    q.qspec_check_status()


def test_sequences_without_tokens_or_positions_and_short_ones():
    """Padded batches: sequences of no tokens (first in their group, too), of no positions, with fewer positions than new tokens."""
    q = lib()
    for many in (1, 30):
        toks = [0, 2 * many, 0, 1, 3, 0, 1]
        kv = [0, 100 + 2 * many, 5, 101, 2, 0, 1]
        bt = ref.Batch(4, toks, kv, 2, 16, 64)
        bt.table[3, :6] = bt.table[1, :6]
        for side in "kv":                          # positions 96 .. 99 of sequence 3 are sequence 1's
            s, d = int(bt.table[1, 6]), int(bt.table[3, 6])
            bt.codes[side][d, :, :4] = bt.codes[side][s, :, :4]
            bt.exps[side][d] = bt.exps[side][s]
        bt.members = [4, 3]
        qt, out, lse = call(q, bt, 4, [100, 50])   # the second group's prefix shrinks to nothing
        check(bt, qt, out, lse)
        q.qspec_check_status()


def test_a_prefix_ends_where_new_tokens_begin():
    q = lib()
    for members, tok in (([3], 2), ([40], 3)):
        bt = shared_batch(9, members, lambda r: tok, [150], lambda r: 0, 1, 32, 64)
        for given in (150, 151, 152, 1000):
            qt, out, lse = call(q, bt, 4, [min(given, bt.table.shape[1] * 32)])
            check(bt, qt, out, lse)
        q.qspec_check_status()


def test_no_prefix_and_single_groups_are_plain_attention():
    q = lib()
    for toks, kv in (([1, 3, 2], [70, 300, 2]), ([20, 40], [500, 333])):
        bt = ref.Batch(6, toks, kv, 2, 64, 128)
        for members, prefix in (([len(toks)], [0]), ([1] * len(toks), [60] * len(toks))):
            bt.members = members
            qt, out, lse = call(q, bt, 8, prefix)
            check(bt, qt, out, lse)
    q.qspec_check_status()


def test_sequences_of_no_group_are_left_as_they_were():
    q = lib()
    for n in (1, 40):
        bt = ref.Batch(8, [n, n, n], [100, 200, 300], 1, 16, 64)
        bt.members = [1]
        cache, batch = bt.gpu(q)
        qt, out, lse = call(q, bt, 2, [10], members=[1])
        check(bt, qt, out, lse, rows=slice(0, n))
        assert bool((out[n:] == 7).all()) and bool((lse[n:] == 7).all())
        # groups that begin behind the first sequence, and groups of none
        pre = q.KVPrefixes(i32_dev([1, 1, 2, 2]), i32_dev([5, 100, 7]), n)
        out, lse = torch.full((3 * n, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((3 * n, 2), 7.0, device=DEV)
        q.qspec_kv_attention_shared(cache, batch, pre, qt.to(DEV), out, q.new_kv_attention_workspace(), lse=lse)
        out, lse = out.double().cpu(), lse.double().cpu()
        check(bt, qt, out, lse, rows=slice(n, 2 * n))
        assert bool((out[:n] == 7).all()) and bool((out[2 * n:] == 7).all()) and bool((lse[2 * n:] == 7).all())
    q.qspec_check_status()


def test_many_groups_and_sequences():
    q = lib()
    members = [2] * 512
    bt = shared_batch(2, members, lambda r: int(r.integers(1, 3)), [40] * 512, lambda r: int(r.integers(0, 6)), 1, 16, 64)
    qt, out, lse = call(q, bt, 2, [40] * 512)
    check(bt, qt, out, lse)
    qt, out, lse = call(q, bt, 2, [40] * 512, max_tok=40)     # the same on the tensor cores
    check(bt, qt, out, lse)
    bt = shared_batch(2, [1024], lambda r: 1, [40], lambda r: int(r.integers(0, 6)), 1, 16, 64)
    qt, out, lse = call(q, bt, 2, [40])
    check(bt, qt, out, lse)
    q.qspec_check_status()


def test_missing_pages_and_bad_numbers_are_reported():
    q = lib()

    def fails(bt, prefix, **more):
        r = call(q, bt, 4, prefix, **more)
        with pytest.raises(q.QSpecError, match="QSPEC_ERR_INVALID_ARG"):
            q.qspec_check_status()
        return r

    for tok in (1, 20):
        def fresh():
            return shared_batch(5, [2, 2], lambda r: tok, [100, 64], lambda r: 20, 1, 16, 64)
        half = slice(2 * tok, None)
        for change in ("kv", "cu", "prefix", "negative", "max_tok", "order", "beyond"):
            bt, prefix, more = fresh(), [100, 64], {}
            members, rows = [2, 2], half
            if change == "kv":
                bt.kv[1] = 16 * bt.table.shape[1] + 1
            elif change == "cu":
                bt.cu[1] = -1
            elif change == "prefix":
                prefix[0] = 16 * bt.table.shape[1] + 1
            elif change == "negative":
                prefix[0] = -1
            elif change == "max_tok":
                bt = shared_batch(5, [3, 2], lambda r: tok, [100, 64], lambda r: 20, 1, 16, 64)
                more["max_tok"], members, rows = 2 * tok, [3, 2], slice(3 * tok, None)
            elif change == "order":
                members, rows = [3, -1], None
            else:
                members, rows = [2, 3], None
            qt, out, lse = fails(bt, prefix, members=members, **({"max_tok": 4 * tok} | more))
            good = fresh() if change in ("kv", "cu") else bt
            if rows is None:
                assert bool((out == 7).all()) and bool((lse == 7).all())
            else:
                check(good, qt, out, lse, rows=rows)
                assert bool((out[:rows.start] == 7).all())
        # a page that is missing: its keys alone are left out, for the whole group where it is the prefix's
        bt = fresh()
        bt.table[0, 2] = bt.n_pages
        qt, out, lse = fails(bt, [100, 64])
        check(fresh(), qt, out, lse, rows=half)
        assert bool(torch.isfinite(out).all())


def test_queries_that_are_not_finite_spoil_their_own_rows():
    q = lib()
    for members in ([3], [30]):
        bt = shared_batch(1, members, lambda r: 1, [100], lambda r: 9, 1, 16, 64)
        qt, _, _ = call(q, bt, 4, [100])
        bad = qt.clone()
        bad[0, 1, 5], bad[2, 3, 0] = math.nan, math.inf
        _, out, lse = call(q, bt, 4, [100], qt=bad)
        assert bool(torch.isnan(out[0, 1]).all()) and bool(torch.isnan(out[2, 3]).all()) and bool(torch.isnan(lse[0, 1]))
        good = torch.ones(bt.T, 4, dtype=torch.bool)
        good[0, 1] = good[2, 3] = False
        want, want_l, tol, tol_l = ref.attention(bt, qt, bt.D ** -0.5)
        assert bool(((out - want).abs() <= tol)[good].all()) and bool(((lse - want_l).abs() <= tol_l)[good].all())
    q.qspec_check_status()


def test_strided_rows_graphs_streams_and_repeats():
    q = lib()
    for tok in (1, 12):
        bt = shared_batch(3, [4, 3], lambda r: tok, [222, 100], lambda r: 30, 2, 32, 64)
        cache, batch = bt.gpu(q)
        pre = q.KVPrefixes(i32_dev([0, 4, 7]), i32_dev([222, 100]), 4 * tok)
        wide = torch.randn(bt.T, 10, 64, device=DEV).to(torch.bfloat16)
        room = torch.full((bt.T, 11, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        lse, ws = torch.empty(bt.T, 8, device=DEV), q.new_kv_attention_workspace()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            q.qspec_kv_attention_shared(cache, batch, pre, wide[:, 1:9], room[:, 2:10], ws, lse=lse)
        torch.cuda.current_stream().wait_stream(side)
        check(bt, wide[:, 1:9].cpu(), room[:, 2:10].double().cpu(), lse.double().cpu())
        assert bool((room[:, :2] == 7).all()) and bool((room[:, 10:] == 7).all())
        first, first_l = room.clone(), lse.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            q.qspec_kv_attention_shared(cache, batch, pre, wide[:, 1:9], room[:, 2:10], ws, lse=lse)
            q.qspec_kv_attention(cache, batch, wide[:, 1:9], room[:, 2:10], ws)      # one workspace for both calls
            q.qspec_kv_attention_shared(cache, batch, pre, wide[:, 1:9], room[:, 2:10], ws, lse=lse)
        for _ in range(3):
            room.fill_(7)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(room, first) and torch.equal(lse, first_l)
        pre.lengths.copy_(i32_dev([130, 0]))       # read when the kernels run
        graph.replay()
        check(bt, wide[:, 1:9].cpu(), room[:, 2:10].double().cpu(), lse.double().cpu())
    q.qspec_check_status()


def test_pages_of_the_prefix_are_looked_up_for_the_first_sequence_alone():
    q = lib()
    for members, tok in (([3], 1), ([4], 20)):
        for prefix in (100, 128, 250):
            bt = shared_batch(prefix, members, lambda r: tok, [prefix], lambda r: 70, 2, 16, 64)
            qt, out, lse = call(q, bt, 8, [prefix])
            bt.table[1:, :prefix // 16] = -5
            _, out2, lse2 = call(q, bt, 8, [prefix])
            q.qspec_check_status()
            assert torch.equal(out, out2) and torch.equal(lse, lse2)
