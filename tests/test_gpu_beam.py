"""Beam selection against the definition in 64 bits: parents and tokens equal, scores within an fp32 rounding.

Scores: fp32 terms 2^((x - m) log2 e) carry a relative error below 2^-21 (the difference, the product and the approximate power, and at
most 15 fp32 additions by trees, 10 more by shuffles), so lse is within 2^-20 absolutely; S is rounded to fp32 once."""
import math

import pytest
import torch

from gpu_util import DEV, lib

pytestmark = pytest.mark.gpu
NEAR = 2.0 ** -19    # candidates of different beams nearer than this may change places


def definition(x, scores, n, done=None, end_tok=0, weights=None):
    """[[(parent, token, S)]] of each sequence, in order, and the weighted S of all candidates in order."""
    B, K, V = x.shape
    out, ranks = [], []
    for b in range(B):
        cand = []
        for k in range(K):
            s = float(scores[b, k])
            w = 1.0 if weights is None else float(weights[b, k])
            if s == -math.inf:
                continue
            if done is not None and int(done[b, k]):
                cand.append((-s * w, k, 0, b * K + k, end_tok, s))
                continue
            z = x[b, k].double().cpu()
            if float(z.max()) == -math.inf:
                continue
            lse = float(torch.logsumexp(z, 0))
            order = torch.sort(z, descending=True, stable=True).indices[:n + 1]
            for i, v in enumerate(order.tolist()):
                if float(z[v]) > -math.inf:
                    S = s + (float(z[v]) - lse)
                    cand.append((-S * w, k, i, b * K + k, v, S))
        cand.sort()
        out.append([c[3:] for c in cand[:n]])
        ranks.append([-c[0] for c in cand])
    return out, ranks


def call(q, x, scores, n, **more):
    B, K, V = x.shape
    parent, tok = (torch.full((B, n), 77, dtype=torch.int32, device=DEV) for _ in range(2))
    score = torch.full((B, n), 7.0, device=DEV)
    ws = more.pop("ws", None)
    q.qspec_beam_select(x, scores, parent, tok, score, q.new_beam_workspace(B, K, V, n) if ws is None else ws, **more)
    return parent.cpu(), tok.cpu(), score.cpu()


def check(got, x, scores, n, **more):
    want, ranks = definition(x, scores, n, **more)
    parent, tok, score = got
    for b, (row, rank) in enumerate(zip(want, ranks)):
        clear = all(abs(p - r) > NEAR or p == r for p, r in zip(rank[:n], rank[1:n + 1]))
        assert clear, "the inputs of a test leave no near ties"
        for i in range(n):
            p, t, S = row[i] if i < len(row) else (-1, -1, -math.inf)
            assert (int(parent[b, i]), int(tok[b, i])) == (p, t), (b, i)
            assert float(score[b, i]) == S or abs(float(score[b, i]) - S) <= 2.0 ** -20 + 2.0 ** -24 * abs(S), (b, i, float(score[b, i]), S)


def inputs(seed, B, K, V, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(B, K, V, generator=g) * 2 * spread).to(torch.bfloat16).to(DEV)
    scores = (-10 + 3 * torch.randn(B, K, generator=g)).to(DEV)
    return x, scores, g


@pytest.mark.parametrize("B,K,V,n", [(1, 1, 2, 1), (1, 2, 3, 6), (3, 4, 999, 4), (2, 5, 32000, 10), (1, 1, 50001, 64), (4, 3, 32761, 3),
                                     (2, 2, 128256, 16), (1, 8, 152064, 17), (2, 32, 4097, 32), (1, 4, 70003, 33), (64, 8, 513, 8), (1, 2, 16, 32)])
def test_against_the_definition(B, K, V, n):
    q = lib()
    for seed in range(2):
        x, scores, _ = inputs(seed + V, B, K, V)
        check(call(q, x, scores, n), x, scores, n)
    q.qspec_check_status()


@pytest.mark.parametrize("V", [1000, 40001, 152064])
def test_finished_beams_weights_and_empty_beams(V):
    q = lib()
    B, K, n = 6, 4, 8
    x, scores, g = inputs(V, B, K, V)
    done = (torch.rand(B, K, generator=g) < 0.4).to(torch.int32).to(DEV)
    weights = (0.2 + torch.rand(B, K, generator=g)).to(DEV)
    scores[0, 1:] = -math.inf                 # the first step: one beam
    done[1] = 1                               # all ended
    scores[2, 0] = -math.inf
    x[3, 2] = -math.inf
    x[4, :, 3:] = -math.inf                   # a grammar that leaves three tokens
    scores[5] = -math.inf                     # nothing at all
    for d, w in ((None, None), (done, None), (None, weights), (done, weights)):
        check(call(q, x, scores, n, done=d, end_tok=-3, weights=w), x, scores, n, done=d, end_tok=-3, weights=w)
    q.qspec_check_status()


@pytest.mark.parametrize("V,n", [(300, 5), (32000, 8), (100003, 64)])
def test_equal_logits_go_to_the_lowest_token(V, n):
    q = lib()
    x = torch.zeros(2, 3, V, dtype=torch.bfloat16, device=DEV)
    x[0, 1] = -0.0
    x[0, 1, ::2] = 0.0                        # -0 and 0 are equal
    x[1, 0] = 3.0
    x[1, 1, V // 2:] = 1.0                    # equal in the later half
    x[1, 2, ::3] = 1.5
    scores = torch.tensor([[-1.0, -2.0, -1.5], [-4.0, -1.0, -2.0]], device=DEV)
    check(call(q, x, scores, n), x, scores, n)
    same = torch.zeros(1, 3, V, dtype=torch.bfloat16, device=DEV)
    got = call(q, same, torch.zeros(1, 3, device=DEV), n)   # equal beams: the lowest beam first
    assert got[0].tolist() == [[0] * n] and got[1].tolist() == [list(range(n))]
    q.qspec_check_status()


def test_sorted_rows_fill_the_candidate_lists():
    """Ascending and descending logits: one thread or one end of the row holds all that counts."""
    q = lib()
    V = 40000
    x = torch.linspace(-30, 30, V).to(torch.bfloat16).to(DEV)
    rows = torch.stack([x, x.flip(0), torch.roll(x, V // 3), x.abs()])[None].contiguous()
    scores = torch.tensor([[-1.0, -2.1, -3.3, -0.7]], device=DEV)
    for n in (1, 16, 40, 64):
        check(call(q, rows, scores, n), rows, scores, n)
    block = torch.full((1, 2, V), -5.0, dtype=torch.bfloat16, device=DEV)  # 4096 large ones behind another, in one thread's share and out of it
    block[0, 0, 1000:5096] = torch.linspace(1, 9, 4096, device=DEV).to(torch.bfloat16)
    block[0, 1, 16:24] = 4.0
    check(call(q, block, scores[:, :2], 24), block, scores[:, :2], 24)
    q.qspec_check_status()


def test_a_vocabulary_of_several_tiles_to_a_chunk():
    q = lib()
    V, K = 2_000_003, 32                      # 16 chunks of four tiles
    x, scores, g = inputs(3, 1, K, V)
    x[0, 5, -1] = 20.0
    x[0, 7, 0] = 21.0
    x[0, 9] = 1.0                             # ties through all tiles
    check(call(q, x, scores, 40), x, scores, 40)
    q.qspec_check_status()


def test_far_scores_and_flat_logits():
    q = lib()
    x, _, _ = inputs(1, 2, 3, 5000, spread=0.0)
    scores = torch.tensor([[-3e4, -3.5e4, -2.5e4], [0.0, 1e3, 2e3]], device=DEV)
    check(call(q, x, scores, 6), x, scores, 6)
    x, _, _ = inputs(2, 2, 3, 5000, spread=1e4)
    check(call(q, x, scores, 6), x, scores, 6)
    q.qspec_check_status()


def test_bad_values_are_reported_and_their_beams_left_out():
    q = lib()
    for change in ("nan", "-nan", "inf", "score nan", "score inf", "weight 0", "weight -1", "weight nan", "weight inf"):
        x, scores, _ = inputs(4, 2, 3, 70001)
        weights = torch.ones(2, 3, device=DEV)
        kind, _, v = change.partition(" ")
        if kind in ("nan", "-nan"):
            x.view(torch.int16)[1, 1, 69999] = 0x7FC1 if kind == "nan" else -1
        elif kind == "inf":
            x[1, 1, 3] = math.inf
        else:
            (scores if kind == "score" else weights)[1, 1] = float(v)
        got = call(q, x, scores, 4, weights=weights)
        with pytest.raises(q.QSpecError, match="QSPEC_ERR_INVALID_ARG"):
            q.qspec_check_status()
        scores[1, 1], weights[1, 1] = -math.inf, 1.0
        check(got, x, scores, 4, weights=weights)


def test_a_workspace_serves_call_after_call_in_a_graph_and_on_another_stream():
    q = lib()
    B, K, V, n = 3, 4, 30000, 4
    ws = q.new_beam_workspace(B, K, V, n)
    x, scores, _ = inputs(8, B, K, V)
    parent, tok = (torch.zeros(B, n, dtype=torch.int32, device=DEV) for _ in range(2))
    score = torch.zeros(B, n, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q.qspec_beam_select(x, scores, parent, tok, score, ws)
    torch.cuda.current_stream().wait_stream(side)
    check((parent.cpu(), tok.cpu(), score.cpu()), x, scores, n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.qspec_beam_select(x, scores, parent, tok, score, ws)
    for seed in (9, 10, 11):
        y, s, _ = inputs(seed, B, K, V)
        x.copy_(y)
        scores.copy_(s)
        graph.replay()
        check((parent.cpu(), tok.cpu(), score.cpu()), x, scores, n)
    q.qspec_check_status()


def test_a_workspace_serves_smaller_shapes_too():
    q = lib()
    ws = q.new_beam_workspace(20, 5, 9000, 10)
    for B, K, V, n in ((20, 5, 9000, 10), (3, 5, 9000, 2), (20, 1, 70, 10), (7, 4, 8191, 5), (20, 5, 9000, 10)):
        x, scores, _ = inputs(B + V, B, K, V)
        check(call(q, x, scores, n, ws=ws), x, scores, n)
    q.qspec_check_status()


@pytest.mark.parametrize("m", [300, 700, 1500, 5000, 20000, 152064])
@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("n", [1, 8, 64])
def test_ever_better_logits(m, rising, n):
    """m logits that rise (or fall) along the row, the rest below them: later ones pass every bound that the earlier ones gave."""
    V = 152064
    x, scores, g = inputs(31 + m, 1, 1, V, 0.5)
    at = torch.randperm(V, generator=g)[:m].sort().values
    ramp = torch.linspace(8, 40, m)
    x[0, 0, at.to(DEV)] = (ramp if rising else ramp.flip(0)).to(torch.bfloat16).to(DEV)
    check(call(lib(), x, scores, n), x, scores, n)
