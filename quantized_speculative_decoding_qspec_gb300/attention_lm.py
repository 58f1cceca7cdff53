"""Speculative decoding of a small attention model on the library's calls.

One decoder layer between an embedding and an output projection, on seeded synthetic weights: 4-bit
linears in both modes, rotary positions, the paged 8-bit cache, attention over it, adjusted logits and
greedy verification, put together as a serving loop uses them:

* a prompt is one pass of all its tokens in W4A16 mode;
* the draft extends every sequence gamma times in W4A4 mode, one token a pass, each pass writing its
  keys behind the sequence;
* one W4A16 pass over the gamma + 1 positions writes them again with the verify mode's keys, and the
  adjusted logits of all positions go to the verify call, position i counting the drafts before it;
* what was rejected is dropped by a smaller length.

Every emitted token is the greedy choice of the W4A16 pass that verified it.  The cache that this pass attends to is not
quite the one that decoding token by token would have left: drafted and rejected tokens may have raised a page's scale, and
the codes of accepted ones below e4m3's normal range were rounded again.  Where two logits are as near as that, the text can
differ from plain W4A16 decoding.

``Beams`` continues each prompt in several beams instead: their sequences share the prompt's pages and, where they go on from
the same beam, its pages too; attention reads a prompt's keys once for all its beams, and a step ends with the choice of
the next beams and their page tables, without a look at anything on the host.

``python -m quantized_speculative_decoding_qspec_gb300.attention_lm`` runs both on one GPU.
"""
from __future__ import annotations

import torch

from . import qspec as q


class AttentionLM:
    """Embedding [V, width], one attention layer (heads_q query heads on heads key heads of dim), output [V, width]."""

    def __init__(self, V=1024, width=512, heads_q=8, heads=2, dim=64, page=16, n_pages=256, seed=0, device="cuda"):
        self.V, self.width, self.heads_q, self.heads, self.dim = V, width, heads_q, heads, dim
        self.device = device
        g = torch.Generator().manual_seed(seed)
        self.E = torch.randn(V, width, generator=g).to(torch.bfloat16).to(device)
        n_qkv = (heads_q + 2 * heads) * dim
        self.linears = {}
        for name, (N, K) in {"qkv": (n_qkv, width), "o": (width, heads_q * dim), "out": (V, width)}.items():
            W = (torch.randn(N, K, generator=g) * K ** -0.5).to(torch.bfloat16).to(device)
            Wp = torch.empty(N, K // 2, dtype=torch.uint8, device=device)
            S = torch.empty(N, K // 128, dtype=torch.float16, device=device)
            q.qspec_pack_weights(W, Wp, S)
            self.linears[name] = (Wp, S)
        self.rotary = q.Rotary(dim, base=10000.0, device=device)
        self.cache = q.new_kv_cache(n_pages, heads, page, dim, device=device)
        self.ws = q.new_kv_attention_workspace(device)
        self._linear_ws = {}

    def _linear(self, name, x, draft_mode):
        Wp, S = self.linears[name]
        M, (N, K) = x.shape[0], (Wp.shape[0], 2 * Wp.shape[1])
        ws = self._linear_ws.get((name, M))
        if ws is None:
            ws = self._linear_ws[name, M] = q.new_linear_workspace(M, N, K, device=self.device)
        y = torch.empty(M, N, dtype=torch.bfloat16, device=self.device)
        (q.qspec_linear_w4a4 if draft_mode else q.qspec_linear_w4a16)(x, Wp, S, y, ws)
        return y

    def forward(self, tok, batch, draft_mode, tree=None, pos=None, prefixes=None):
        """Logits [T, V] of the new tokens tok int32 [T] (sequence after sequence), whose keys join the cache.  prefixes: what
        the sequences share, or None."""
        T, hq, hk, d = tok.numel(), self.heads_q, self.heads, self.dim
        x = torch.empty(T, self.width, dtype=torch.bfloat16, device=self.device)
        q.qspec_gather_rows(self.E, tok, x)
        qkv = self._linear("qkv", x, draft_mode).view(T, hq + 2 * hk, d)
        # queries, keys and values are slices of one projection's rows; the queries rotate in place
        qs, ks, vs = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        q.qspec_kv_append(self.cache, batch, ks, vs, rotary=self.rotary, q=qs, pos=pos)
        att = torch.empty(T, hq, d, dtype=torch.bfloat16, device=self.device)
        if prefixes is None:
            q.qspec_kv_attention(self.cache, batch, qs, att, self.ws, tree=tree)
        else:
            q.qspec_kv_attention_shared(self.cache, batch, prefixes, qs, att, self.ws, tree=tree)
        return self._linear("out", x + self._linear("o", att.view(T, hq * d), draft_mode), draft_mode)


def _take(cache):
    """The cache's pages are the caller's from now on; what shares them out beside it keeps the token."""
    cache.claim = claim = object()
    return claim


def _still_has(cache, claim):
    if getattr(cache, "claim", None) is not claim:
        raise ValueError("the cache's pages are another serving loop's or beam search's by now")


class Server:
    """B sequences decoded together: gamma drafted tokens and one verify pass an iteration.  It takes the model's cache: a serving
    loop or beam search that had it before makes no step any more.

    penalties: (repetition, frequency, presence) of every sequence, or None; allowed: int32 [ceil(V/32)]
    words of the tokens that may be emitted, or None.  A prompt has 1 to max_len tokens; step() refuses once a
    sequence has more than max_len in the cache, as its history and pages end behind one step more.
    """

    def __init__(self, model, prompts, gamma=3, max_len=256, penalties=None, allowed=None):
        if not prompts or gamma < 1:
            raise ValueError("at least one prompt and one drafted token a step")
        for p in prompts:
            if not 1 <= len(p) <= max_len:
                raise ValueError(f"a prompt has 1 to {max_len} tokens, got {len(p)}")
        dev, B = model.device, len(prompts)
        self.model, self.B, self.gamma, self.max_len = model, B, gamma, max_len
        self.longest = max(len(p) for p in prompts)  # cached positions of the longest sequence, at most
        self.max_pages = -(-(max_len + gamma + 1) // model.cache.page)
        if B * self.max_pages > model.cache.k.shape[0]:
            raise ValueError("the cache has too few pages")
        i32 = dict(dtype=torch.int32, device=dev)
        self.pages = torch.randperm(B * self.max_pages, device=dev).to(torch.int32).view(B, self.max_pages)
        self.kv_len = torch.zeros(B, **i32)
        self.prompt_len = torch.tensor([len(p) for p in prompts], **i32)
        self.hist = torch.zeros(B, max_len + gamma + 2, **i32)
        self.hist_len = self.prompt_len.clone()
        for b, p in enumerate(prompts):
            self.hist[b, :len(p)] = torch.tensor(p, **i32)
        self.pen = None if penalties is None else torch.tensor([penalties] * B, dtype=torch.float32, device=dev)
        self.allowed = allowed
        self.vws = q.new_verify_workspace(B, gamma, model.V, device=dev)
        self.n, self.out = torch.zeros(B, **i32), torch.zeros(B, gamma + 1, **i32)
        self.rows = torch.arange(B, device=dev)
        self.claim = _take(model.cache)
        self._prefill(prompts)

    def _batch(self, n):
        """n new tokens of every sequence; the lengths are read from kv_len when the kernels run."""
        cu = torch.arange(0, (self.B + 1) * n, n, dtype=torch.int32, device=self.model.device)
        return q.KVBatch(cu, self.kv_len, self.pages, n)

    def _adjust(self, logits, draft=None, hist_len=None):
        rows = logits.shape[1]
        mask = None if self.allowed is None else self.allowed.expand(self.B, rows, -1).contiguous()
        q.qspec_logits_adjust(logits, logits, draft_tok=draft, hist=self.hist, hist_len=self.hist_len if hist_len is None else hist_len,
                              prompt_len=self.prompt_len, penalties=self.pen, mask=mask)
        return logits

    def _prefill(self, prompts):
        lens = [len(p) for p in prompts]
        ends = torch.tensor(lens).cumsum(0)
        cu = torch.cat([torch.zeros(1, dtype=torch.int64), ends]).to(torch.int32).to(self.model.device)
        self.kv_len.copy_(self.prompt_len)
        tok = torch.cat([self.hist[b, :n] for b, n in enumerate(lens)])
        logits = self.model.forward(tok, q.KVBatch(cu, self.kv_len, self.pages, max(lens)), draft_mode=False)
        last = logits[(ends - 1).to(logits.device)].view(self.B, 1, -1).contiguous()
        tok = torch.empty(self.B, dtype=torch.int32, device=self.model.device)
        q.qspec_select_tokens(self._adjust(last)[:, 0].contiguous(), tok)
        self.hist[self.rows, self.hist_len.long()] = tok
        self.hist_len += 1

    def step(self):
        """One iteration; returns the emitted tokens [B, gamma + 1] (-1 behind the accepted ones)."""
        m, B, gamma = self.model, self.B, self.gamma
        if self.longest > self.max_len:              # the bound first, the lengths only when it is reached
            self.longest = int(self.kv_len.max())
            if self.longest > self.max_len:
                raise ValueError(f"a sequence has {self.longest} positions in the cache, beyond max_len {self.max_len}")
        self.longest += gamma + 1
        _still_has(m.cache, self.claim)
        base, length = self.kv_len.clone(), self.hist_len.clone()  # the last token of hist is not in the cache yet
        tokens = torch.empty(B, gamma + 1, dtype=torch.int32, device=m.device)
        tokens[:, 0] = self.hist[self.rows, (length - 1).long()]
        one = self._batch(1)
        for i in range(gamma):
            self.kv_len += 1
            logits = self._adjust(m.forward(tokens[:, i].contiguous(), one, draft_mode=True).view(B, 1, m.V),
                                  hist_len=length + i)
            nxt = torch.empty(B, dtype=torch.int32, device=m.device)
            q.qspec_select_tokens(logits.view(B, m.V), nxt)
            tokens[:, i + 1] = nxt
            self.hist[self.rows, (length + i).long()] = nxt
        self.kv_len.copy_(base + gamma + 1)
        logits = m.forward(tokens.view(-1), self._batch(gamma + 1), draft_mode=False).view(B, gamma + 1, m.V)
        draft = tokens[:, 1:].contiguous()
        q.qspec_verify_greedy(self._adjust(logits, draft=draft), draft, self.n, self.out, self.vws)
        # keep the accepted positions; the emitted token that follows them is fed next time
        self.kv_len.copy_(base + self.n + 1)
        self.hist.scatter_(1, (length[:, None] + torch.arange(gamma + 1, device=m.device)).long(), self.out.clamp(min=0))
        self.hist_len.copy_(length + self.n + 1)
        return self.out


class Beams:
    """Beam search: `beams` continuations of each prompt, by summed log probability.

    end_tok ends a beam, which then stays among the best by its score alone; beams compare by their score divided by the length
    of what they added to the power of `length_power`.  A prompt has 1 to max_len tokens; max_new tokens are added at most.
    tokens [B, beams, max_new] and scores [B, beams] are best first.  The search takes the model's cache, with all its pages free:
    a serving loop or beam search that had it before makes no step any more.
    """

    def __init__(self, model, prompts, beams=4, max_len=256, max_new=64, end_tok=0, length_power=0.0):
        if not prompts or beams < 1 or max_new < 1:
            raise ValueError("at least one prompt, one beam and one new token")
        for p in prompts:
            if not 1 <= len(p) <= max_len:
                raise ValueError(f"a prompt has 1 to {max_len} tokens, got {len(p)}")
        if not 0 <= end_tok < model.V:
            raise ValueError("end_tok must be a token")
        page, dev = model.cache.page, model.device
        B, K = len(prompts), beams
        # a prompt's pages once, and of each beam its own: those of its new tokens and the page that they begin in, twice while they move
        need = sum(-(-len(p) // page) for p in prompts) + 2 * B * K * (-(-max_new // page) + 1)
        if need > model.cache.k.shape[0]:
            raise ValueError(f"the cache has too few pages: {model.cache.k.shape[0]} of {need}")
        self.model, self.B, self.K, self.end_tok, self.max_new, self.power = model, B, K, end_tok, max_new, length_power
        i32 = dict(dtype=torch.int32, device=dev)
        width = -(-(max_len + max_new) // page)
        self.tables = [torch.zeros(B * K, width, **i32) for _ in range(2)]
        self.refs = torch.zeros(model.cache.k.shape[0], **i32)
        self.copies = [torch.zeros(B * K, **i32) for _ in range(3)]
        self.left = torch.zeros(1, **i32)
        self.prompt_len = torch.tensor([len(p) for p in prompts], **i32)
        self.length = self.prompt_len.repeat_interleave(K)             # cached positions of each beam
        self.tokens = torch.full((B, K, max_new), -1, **i32)
        self.parent, self.tok = torch.zeros(B, K, **i32), torch.zeros(B, K, **i32)
        self.score, self.done, self.added = torch.zeros(B, K, device=dev), torch.zeros(B, K, **i32), torch.zeros(B, K, **i32)
        self.bws = q.new_beam_workspace(B, K, model.V, K, device=dev)
        self.cu = torch.arange(B * K + 1, **i32)
        self.prefixes = q.KVPrefixes(torch.arange(0, B * K + 1, K, **i32), self.prompt_len, K)
        self.steps, self.closed = 0, False
        self.claim = _take(model.cache)
        self._prefill(prompts)

    def _pages(self, lengths, parent, keep, need):
        """The next page tables from the present ones, whose first rows hold `lengths` positions, and the copies that they ask for."""
        old, new = self.tables
        src, dst, size = self.copies
        q.qspec_kv_pages(old[:lengths.numel()], lengths, keep, need, self.refs, self.model.cache.page, new[:keep.numel()], self.refs,
                         src[:keep.numel()], dst[:keep.numel()], size[:keep.numel()], self.left, parent=parent)
        q.qspec_kv_copy_pages(self.model.cache, src[:keep.numel()], dst[:keep.numel()], lengths=size[:keep.numel()])
        self.tables.reverse()

    def _prefill(self, prompts):
        B, K, dev = self.B, self.K, self.model.device
        ends = torch.tensor([len(p) for p in prompts]).cumsum(0)
        cu = torch.cat([torch.zeros(1, dtype=torch.int64), ends]).to(torch.int32).to(dev)
        none = torch.full((B,), -1, dtype=torch.int32, device=dev)
        self._pages(none[:0], none, torch.zeros_like(none), self.prompt_len)
        tok = torch.tensor([t for p in prompts for t in p], dtype=torch.int32, device=dev)
        batch = q.KVBatch(cu, self.prompt_len, self.tables[0][:B], max(len(p) for p in prompts))
        logits = self.model.forward(tok, batch, draft_mode=False)
        last = logits[(ends - 1).to(dev)].view(B, 1, -1).contiguous()
        ws = q.new_beam_workspace(B, 1, self.model.V, K, device=dev)
        q.qspec_beam_select(last, torch.zeros(B, 1, device=dev), self.parent, self.tok, self.score, ws)
        self._fork(self.prompt_len)                                    # the old rows are the prompts

    def _fork(self, lengths):
        """The chosen beams go on from their parents' pages (the first rows, of these lengths), with room for one token more.  A beam that
        nothing continues (parent -1: the prompt's logits are not finite) has no pages and no positions, so nothing is written for it."""
        parent, n = self.parent.view(-1), self.steps
        at, lives = parent.long().clamp(min=0), parent >= 0
        keep = torch.where(lives, lengths[at], 0)
        self.length = keep + lives.to(torch.int32)
        self._pages(lengths, parent, keep, self.length)
        if n > 0:                                                      # (parents are rows of the beams before)
            moved = torch.empty_like(self.tokens.view(-1, self.max_new))
            q.qspec_gather_rows(self.tokens.view(-1, self.max_new), parent.clamp(min=0), moved)
            self.tokens = torch.where(lives[:, None], moved, -1).view_as(self.tokens)
            self.done, self.added = self.done.view(-1)[at].view_as(self.done), self.added.view(-1)[at].view_as(self.added)
        self.tokens[:, :, n] = torch.where(self.done != 0, -1, self.tok)
        self.added += (self.done == 0).to(torch.int32)
        self.done |= (self.tok == self.end_tok).to(torch.int32)
        self.steps += 1

    def step(self):
        """One token more for every beam that has not ended."""
        if self.closed:
            raise ValueError("the search is closed")
        if self.steps >= self.max_new:
            raise ValueError(f"the beams have {self.max_new} tokens")
        _still_has(self.model.cache, self.claim)
        B, K, V = self.B, self.K, self.model.V
        batch = q.KVBatch(self.cu, self.length, self.tables[0], 1)
        logits = self.model.forward(self.tok.view(-1), batch, draft_mode=False, prefixes=self.prefixes).view(B, K, V)
        # an ended beam's length stays as it is, the others' grows
        weights = (self.added + (self.done == 0).to(torch.int32)).float() ** -self.power if self.power else None
        parent, tok, score = torch.empty_like(self.parent), torch.empty_like(self.tok), torch.empty_like(self.score)
        q.qspec_beam_select(logits, self.score, parent, tok, score, self.bws, done=self.done, end_tok=self.end_tok, weights=weights)
        self.parent, self.tok, self.score = parent, tok, score
        self._fork(self.length)

    def close(self):
        """Gives all pages back; no step can follow."""
        if self.closed:
            return
        self.closed = True
        none = self.length[:0]
        q.qspec_kv_pages(self.tables[0], self.length, none, none, self.refs, self.model.cache.page, self.tables[1][:0], self.refs, none,
                         none, none, self.left)


def main():
    model = AttentionLM()
    prompts = [[1, 2, 3, 4, 5], list(range(100, 140)), [7]]
    server = Server(model, prompts, gamma=3, max_len=128, penalties=(1.1, 0.2, 0.1))
    accepted = []
    for _ in range(20):
        server.step()
        accepted.append(server.n.float().mean().item())
    q.qspec_check_status(server.vws)
    for b, p in enumerate(prompts):
        n = int(server.hist_len[b])
        print(f"sequence {b}: {n - len(p)} tokens, cache length {int(server.kv_len[b])}: {server.hist[b, len(p):n].tolist()}")
    print(f"accepted drafts per iteration: {sum(accepted) / len(accepted):.2f} of {server.gamma}")
    search = Beams(model, prompts, beams=4, max_len=128, max_new=12, length_power=0.6)
    for _ in range(11):
        search.step()
    q.qspec_check_status()
    for b in range(len(prompts)):
        print(f"beams of prompt {b}: " + ", ".join(f"{float(search.score[b, k]):.2f} {search.tokens[b, k, :6].tolist()}" for k in range(4)))


if __name__ == "__main__":
    main()
