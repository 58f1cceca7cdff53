"""Beam selection where sums round alike: equal (weighted) S in the order of the beams, a beam's own in the order of its logits, then
of its tokens.  Scores are so large, or weights and logits so small, that a beam's S are the same number in fp64, or there is one beam
with a score of its own; so what is expected does not depend on how the logarithm rounds."""
import math

import pytest
import torch

from gpu_util import DEV, lib

pytestmark = pytest.mark.gpu
LOWEST = torch.finfo(torch.float32).min


def best_first(row, n):
    z = row.double().cpu()
    return [t for t in torch.sort(z, descending=True, stable=True).indices[:n].tolist() if float(z[t]) > -math.inf]


def call(q, x, scores, n, **more):
    B, K, V = x.shape
    parent, tok = (torch.full((B, n), 77, dtype=torch.int32, device=DEV) for _ in range(2))
    score = torch.full((B, n), 7.0, device=DEV)
    q.qspec_beam_select(x, scores, parent, tok, score, q.new_beam_workspace(B, K, V, n), **more)
    q.qspec_check_status()
    return parent.tolist(), tok.tolist(), score.tolist()


def logits(seed, *shape, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * spread).to(torch.bfloat16).to(DEV)


@pytest.mark.parametrize("score", [-10.0, -1e9, -1e14, -1e15, -1e16, -1e30, LOWEST])
@pytest.mark.parametrize("V", [2000, 32000, 152064])
@pytest.mark.parametrize("n", [1, 8, 64])
def test_one_beam_keeps_the_order_of_its_logits(score, V, n):
    q = lib()
    for seed, spread in ((1, 2.0), (2, 0.01), (3, 1e-30)):
        x = logits(seed + V, 2, 1, V, spread=spread)
        parent, tok, got = call(q, x, torch.full((2, 1), score, device=DEV), n)
        for b in range(2):
            assert parent[b] == [b] * n and tok[b] == best_first(x[b, 0], n), seed
            if score <= -1e9:
                assert got[b] == [torch.tensor(score, dtype=torch.float32).item()] * n


@pytest.mark.parametrize("score", [-1e30, LOWEST])
@pytest.mark.parametrize("n", [1, 8, 64])
def test_equal_sums_go_by_beam_then_by_logit(score, n):
    """Beams of one huge score: the first of them that has logits left gives its best ones, then the next."""
    q = lib()
    V, K = 50001, 6
    x = logits(n, 3, K, V)
    x[1, 0, 5:] = -math.inf                       # five tokens, then the next beam's
    x[1, 1, ::2] = -math.inf
    x[2, :, 7:-7] = -math.inf                     # fourteen tokens a beam, at both ends of the row
    scores = torch.full((3, K), score, device=DEV)
    scores[1, 2] = -math.inf
    done = torch.zeros(3, K, dtype=torch.int32, device=DEV)
    done[2, 1] = 1                                # offers itself, between beams 0 and 2
    for d in (None, done):
        parent, tok, _ = call(q, x, scores, n, done=d, end_tok=9)
        for b in range(3):
            want = []
            for k in range(K):
                if float(scores[b, k]) == -math.inf:
                    continue
                if d is not None and int(d[b, k]):
                    want.append((b * K + k, 9))
                else:
                    want += [(b * K + k, t) for t in best_first(x[b, k], n)]
            assert list(zip(parent[b], tok[b])) == want[:n], b


@pytest.mark.parametrize("n", [4, 32])
def test_live_beams_before_unused_ones(n):
    """Beams that are not in use yet have the lowest score: what they offer comes behind all else, in the order of their logits."""
    q = lib()
    V, K = 32000, 4
    x = logits(n, 1, K, V)
    x[0, 0, 3:] = -math.inf                       # the live beam has three tokens
    scores = torch.tensor([[-4.0, LOWEST, -1e30, LOWEST]], device=DEV)
    parent, tok, score = call(q, x, scores, n)
    want = [(0, t) for t in best_first(x[0, 0], n)] + [(2, t) for t in best_first(x[0, 2], n)]
    assert list(zip(parent[0], tok[0])) == want[:n]
    assert all(math.isfinite(s) for s in score[0])


@pytest.mark.parametrize("weight", [1e-38, 1.0, 1e38])
def test_weighted_sums_that_round_alike(weight):
    """Logits of about 2^-60 behind a sum of logarithm 10: their S are one number, with any weight."""
    q = lib()
    V, K, n = 32000, 3, 16
    x = logits(7, 2, K, V, spread=2.0 ** -60)
    scores = torch.tensor([[-3.0, -2.0, -1.0], [-1.0, -2.0, -3.0]], device=DEV)
    weights = torch.full((2, K), weight, device=DEV)
    parent, tok, _ = call(q, x, scores, n, weights=weights)
    for b, k in ((0, 2), (1, 0)):
        assert parent[b] == [b * K + k] * n and tok[b] == best_first(x[b, k], n)
