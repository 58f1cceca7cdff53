"""Beam search and tree decoding on the attention model: selection, page tables, copies, attention over shared prefixes and
compacted paths run together as a serving loop uses them."""
import math

import numpy as np
import pytest
import torch

import kv_ref as ref
from gpu_util import DEV, i32_dev, lib
from quantized_speculative_decoding_qspec_gb300 import attention_lm as lm

pytestmark = pytest.mark.gpu


def one_pass(model, q, seq):
    """Log probabilities [n, V] behind each token of seq, by plain attention over a cache of its own."""
    page = model.cache.page
    cache, model.cache = model.cache, q.new_kv_cache(-(-len(seq) // page), model.heads, page, model.dim)
    pages = torch.arange(model.cache.k.shape[0], dtype=torch.int32, device=DEV)[None]
    batch = q.KVBatch(i32_dev([0, len(seq)]), i32_dev([len(seq)]), pages, len(seq))
    logits = model.forward(i32_dev(seq), batch, draft_mode=False)
    model.cache = cache
    return torch.log_softmax(logits.double(), -1).cpu(), float(logits.float().std())


@pytest.mark.parametrize("beams,page,new,power", [(4, 16, 20, 0.0), (3, 64, 12, 0.7), (8, 32, 9, 0.0), (1, 16, 6, 0.0)])
def test_beams_are_scored_by_the_models_probabilities(beams, page, new, power):
    q = lib()
    V = 512
    model = lm.AttentionLM(V=V, width=256, heads_q=4, heads=2, dim=64, page=page, n_pages=160, seed=5)
    g = torch.Generator().manual_seed(6)
    prompts = [torch.randint(0, V, (n,), generator=g).tolist() for n in (70, 1, page)]
    search = lm.Beams(model, prompts, beams=beams, max_len=80, max_new=new, end_tok=7, length_power=power)
    for _ in range(new - 1):
        search.step()
    q.qspec_check_status()
    with pytest.raises(ValueError, match="have"):
        search.step()
    # the counts are those of the tables, and no page that a beam writes in is another's
    refs, table, length = search.refs.cpu().tolist(), search.tables[0].cpu().tolist(), search.length.cpu().tolist()
    want = [0] * len(refs)
    for row, n in zip(table, length):
        for p in row[:-(-n // page)]:
            want[p] += 1
    assert refs == want and int(search.left) == want.count(0)
    assert all(want[row[(n - 1) // page]] == 1 for row, n in zip(table, length))
    tokens, scores = search.tokens.cpu(), search.score.cpu()
    for b, p in enumerate(prompts):
        rows = [tuple(t for t in tokens[b, k].tolist() if t >= 0) for k in range(beams)]
        assert len(set(rows)) == beams                             # beams differ
        ranks = []
        for k, row in enumerate(rows):
            assert 7 not in row[:-1] and (len(row) == new or row[-1] == 7)
            logp, std = one_pass(model, q, list(p) + list(row))
            total = sum(float(logp[len(p) - 1 + i, t]) for i, t in enumerate(row))
            # the two passes round alike but for the order of sums and the codes of pages that grew: a few percent of the
            # logits' spread for each token
            assert abs(float(scores[b, k]) - total) <= 0.05 * std * len(row), (b, k)
            ranks.append(float(scores[b, k]) * (len(row) ** -power if power else 1.0))
        assert ranks == sorted(ranks, reverse=True)
    search.close()
    q.qspec_check_status()
    assert int(search.refs.abs().sum()) == 0 and int(search.left) == len(refs)


def test_one_beam_is_greedy_decoding():
    """A single beam's tokens are the largest logits of one pass over what it wrote, up to the rounding of the two passes."""
    q = lib()
    model = lm.AttentionLM(V=512, width=256, heads_q=4, heads=2, dim=64, page=16, n_pages=64, seed=9)
    prompt = list(range(40, 75))
    search = lm.Beams(model, [prompt], beams=1, max_len=40, max_new=16, end_tok=3)
    for _ in range(15):
        search.step()
    q.qspec_check_status()
    row = [t for t in search.tokens[0, 0].tolist() if t >= 0]
    logp, std = one_pass(model, q, prompt + row)
    for i, t in enumerate(row):
        assert float(logp[len(prompt) - 1 + i, t]) >= float(logp[len(prompt) - 1 + i].max()) - 0.1 * std


def test_a_tree_is_verified_and_its_path_compacted():
    """Two prompts, a tree of candidates each: verified in one pass, the accepted path compacted, and what follows it decoded as from a
    cache that held the path alone."""
    q = lib()
    V, page = 512, 16
    model = lm.AttentionLM(V=V, width=256, heads_q=4, heads=2, dim=64, page=page, n_pages=64, seed=3)
    g = torch.Generator().manual_seed(2)
    prompts = [torch.randint(0, V, (n,), generator=g).tolist() for n in (30, 14)]
    B, T = 2, 9
    # the model's own greedy continuations, hidden among wrong candidates: nodes 1, 4, 6 (then 7 of the second prompt)
    good = [[], []]
    for b, p in enumerate(prompts):
        seq = list(p)
        for _ in range(6):
            logp, _ = one_pass(model, q, seq)
            seq.append(int(logp[-1].argmax()))
        good[b] = seq[len(p):]
    path = [[1, 4, 6], [1, 4, 6, 7]]
    parent = [[-1, -1, 1, 1, 1, 4, 4, 6, 6]] * B
    tok = [[(good[b][0] + 1 + j) % V for j in range(T)] for b in range(B)]
    for b in range(B):
        for i, j in enumerate(path[b]):
            tok[b][j] = good[b][1 + i]                             # (good[0] is fed before the tree)
        for j in range(T):
            if j not in path[b] and tok[b][j] in good[b]:
                tok[b][j] = next(t for t in range(V) if t not in good[b])
    words, depth = [], []
    for b in range(B):
        anc, dep = [1], [0]                                        # bit 0: the token before the tree
        for j in range(T):
            p = parent[b][j]
            anc.append((anc[p + 1] if p >= 0 else 1) | 1 << (j + 1))
            dep.append(dep[p + 1] + 1 if p >= 0 else 1)
        words += anc
        depth += dep
    tables = torch.arange(2 * 6, dtype=torch.int32, device=DEV).view(2, 6)
    lens = [len(p) for p in prompts]
    cu = i32_dev([0] + list(np.cumsum(lens)))
    model.forward(i32_dev(prompts[0] + prompts[1]), q.KVBatch(cu, i32_dev(lens), tables, max(lens)), draft_mode=False)
    new = T + 1
    batch = q.KVBatch(i32_dev([0, new, 2 * new]), i32_dev([n + new for n in lens]), tables, new)
    fed = i32_dev([t for b in range(B) for t in [good[b][0]] + tok[b]])
    pos = i32_dev([lens[i // new] + d for i, d in enumerate(depth)])
    tree = torch.tensor(words, dtype=torch.int64, device=DEV)
    logits = model.forward(fed, batch, draft_mode=False, tree=tree, pos=pos).view(B, new, V)
    n, out, nodes = (torch.zeros(*s, dtype=torch.int32, device=DEV) for s in ((B,), (B, T + 1), (B, T)))
    ws = q.new_tree_workspace(B, T, V)
    q.qspec_verify_tree_greedy(logits, i32_dev(tok), i32_dev(parent), n, out, ws, accept_nodes=nodes)
    q.qspec_kv_compact(model.cache, batch, nodes, n, first=1)
    q.qspec_check_status(ws)
    assert n.tolist() == [3, 4]
    for b in range(B):
        assert nodes[b, :len(path[b])].tolist() == path[b] and out[b, :len(path[b]) + 1].tolist()[:-1] == good[b][1:1 + len(path[b])]
        # the cache now holds prompt, the first token and the path: the values of one pass over them
        seq = prompts[b] + good[b][:1 + len(path[b])]
        kept, model.cache = model.cache, q.new_kv_cache(6, 2, page, 64)
        alone = q.KVBatch(i32_dev([0, len(seq)]), i32_dev([len(seq)]), torch.arange(6, dtype=torch.int32, device=DEV)[None], len(seq))
        model.forward(i32_dev(seq), alone, draft_mode=False)
        for side in "kv":
            one = kept.values(side)[tables[b].long()].permute(1, 0, 2, 3).reshape(2, -1, 64)[:, :len(seq)]
            two = model.cache.values(side).permute(1, 0, 2, 3).reshape(2, -1, 64)[:, :len(seq)]
            assert float((one - two).norm()) <= 2 * ref.E4M3 * float(two.norm())
        model.cache = kept
    # and decoding goes on behind it
    after = i32_dev([lens[b] + 2 + len(path[b]) for b in range(B)])
    last = i32_dev([int(out[b, len(path[b])]) for b in range(B)])
    logits = model.forward(last, q.KVBatch(i32_dev([0, 1, 2]), after, tables, 1), draft_mode=False)
    for b in range(B):
        logp, std = one_pass(model, q, prompts[b] + good[b][:1 + len(path[b])] + [int(last[b])])
        t = int(logits[b].argmax())
        assert float(logp[-1, t]) >= float(logp[-1].max()) - 0.1 * std
    q.qspec_check_status()
    assert math.isfinite(float(logits.float().sum()))
