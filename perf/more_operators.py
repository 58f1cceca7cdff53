"""What several continuations of one prompt need beside the decode step, as measured cases.

Four operators, one pass each:

* beam    -- the best n of a sequence's beams times vocabulary, by summed log probabilities: parents,
             tokens and scores of the next beams;
* fork    -- the page tables of the next step: rows take over their parents' pages, pages that two
             rows would write are copied (in every layer's cache), room for the next token is taken
             from the free pages, pages that nobody holds are free again;
* compact -- the accepted path of a candidate tree moved behind the committed tokens of the paged
             cache of e4m3 codes, in every layer's cache;
* shared  -- causal attention over that cache for sequences that share a long prefix, which is
             computed once for all the sequences of a group.

``own`` False: the plain form, elementary torch operations in fp32 (fp64 for the log probabilities).
``own`` True: the calls a user makes of the library.  Head counts, page sizes, vocabularies and draft lengths are those
of the decode shapes that the benchmark and the tests use (4096-wide layers with 32 heads and 8 key
heads of 128, 8192-wide ones with 64 and 8; vocabularies of 32000, 128256 and 152064), or generic.
"""
import math

import numpy as np
import torch

own = False

EXP_MIN, EXP_MAX = -40, 40


# ---------------------------------------------------------------------------------------- cases

def listed():
    sh = {"op": "shared", "dim": 128, "page": 64, "ragged": False}
    fk = {"op": "fork", "heads": 8, "dim": 128, "page": 64}
    return [
        # one sequence's four beams: the smallest selection, where latency counts
        {"name": "beam_one", "op": "beam", "B": 1, "beams": 4, "V": 32000, "n": 4, "ends": False},
        # a served batch, twice as many candidates as beams, finished beams and length weights
        {"name": "beam_serve", "op": "beam", "B": 16, "beams": 4, "V": 128256, "n": 8, "ends": True},
        # a large batch with eight beams
        {"name": "beam_batch", "op": "beam", "B": 64, "beams": 8, "V": 152064, "n": 8, "ends": True},
        # one sequence's four beams take up their parents' pages
        dict(fk, name="fork_one", groups=1, per=4, prompt=1500, made=37, layers=1),
        # a batch of 64 prompts with four beams, long prompts in shared pages
        dict(fk, name="fork_batch", groups=64, per=4, prompt=4096, made=75, layers=1),
        # the same step for all layers of a model at once, small pages
        dict(fk, name="fork_layers", groups=8, per=4, prompt=600, made=101, layers=32, page=16),
        # trees of 31 candidates, heads of 64, small pages: one layer
        {"name": "compact_tree", "op": "compact", "B": 8, "nodes": 31, "kv": 2049, "heads": 16, "dim": 64, "page": 16, "layers": 1},
        # trees of 63 candidates of 64 sequences, 32 layers
        {"name": "compact_layers", "op": "compact", "B": 64, "nodes": 63, "kv": 300, "heads": 8, "dim": 128, "page": 64, "layers": 32},
        # four beams of one prompt, one token each
        dict(sh, name="shared_beams", groups=1, per=4, tok=1, prefix=2049, suffix=100, hq=32, hk=8),
        # 16 prompts with four continuations each, draft length 3
        dict(sh, name="shared_verify", groups=16, per=4, tok=4, prefix=6001, suffix=300, hq=32, hk=8),
        # 64 samples of one long prompt, 8 query heads to a key head
        dict(sh, name="shared_samples", groups=1, per=64, tok=1, prefix=32768, suffix=512, hq=64, hk=8),
        # three system prompts under 128 conversations of different lengths, up to 4 tokens each
        dict(sh, name="shared_system", groups=3, per=43, tok=4, prefix=16384, suffix=2000, hq=32, hk=8, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["beam", "fork", "compact", "shared", "shared", "shared"])
    if op == "beam":
        B, K = _log(rng, 1, 64), rng.choice([1, 2, 3, 4, 5, 8])
        return {"op": op, "B": B, "beams": K, "V": rng.choice([32000, 50001, 128256, 152064]),
                "n": rng.choice([K, 2 * K]) if B < 64 else K, "ends": rng.random() < 0.6}
    heads, dim, page = rng.choice([2, 8, 16]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    layers = rng.choice([1, 1, 2, 8, 32])
    if op == "fork":
        per, made = rng.randint(2, 8), _log(rng, 1, 300)
        row = layers * heads * dim * 2  # bytes of a token
        most = max(1, (1 << 29) // (row * (per * (made + 2 * page))))
        groups = _log(rng, 1, min(64, most))
        prompt = _log(rng, 3, max(3, min(8192, (1 << 29) // (row * groups))))
        return {"op": op, "groups": groups, "per": per, "prompt": prompt, "made": made, "layers": layers, "heads": heads,
                "dim": dim, "page": page}
    if op == "compact":
        B, nodes = _log(rng, 1, 64), rng.randint(2, 64)
        kv = _log(rng, nodes + 1, max(nodes + 1, min(8192, (1 << 29) // (layers * heads * dim * 2 * B))))
        return {"op": op, "B": B, "nodes": nodes, "kv": kv, "heads": heads, "dim": dim, "page": page, "layers": layers}
    hk, g = rng.choice([(8, 4), (8, 8), (8, 1), (2, 7), (1, 8)])
    groups = _log(rng, 1, 16)
    per = _log(rng, 1, 128 // groups)
    tok = rng.choice([1, 1, rng.randint(2, 8), rng.randint(9, 40)])
    rows = groups * per * tok * hk * g
    prefix = _log(rng, 16, max(64, min(32768, 262144 // groups, (1 << 29) // rows)))
    suffix = _log(rng, tok, max(tok, min(4096, 131072 // (groups * per), (1 << 28) // rows)))
    return {"op": op, "groups": groups, "per": per, "tok": tok, "prefix": prefix, "suffix": suffix, "hq": hk * g, "hk": hk,
            "dim": dim, "page": page, "ragged": rng.random() < 0.5}


# ---------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 29)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def _block_exp(amax):
    """The smallest e with amax <= 448 * 2^e, within the limits."""
    m, k = torch.frexp(amax)                       # amax = m * 2^k, m in [0.5, 1)
    e = torch.where(m > 0.875, k - 8, k - 9)       # 448 = 0.875 * 2^9
    return torch.where(amax > 0, e, torch.full_like(e, EXP_MIN)).clamp(EXP_MIN, EXP_MAX)


def _codes(x, e):
    """fp32 values [..., P, D] under the scales 2^e [...] as e4m3 codes."""
    return (x * torch.exp2(-e.float())[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _values(codes, exps):
    return codes.view(torch.float8_e4m3fn).float() * torch.exp2(exps.float())[..., None, None]


def _fill(g, layers, pages, heads, page, dim):
    """Caches as earlier steps left them (one page more than the caches have, where plain indexing puts what nobody wants)."""
    codes = torch.empty(layers, pages + 1, heads, page, dim, dtype=torch.uint8, device="cuda")
    exps = torch.empty(layers, pages + 1, heads, dtype=torch.int8, device="cuda")
    ch = torch.ones(heads, 1, dim, device="cuda")
    ch[..., torch.randint(0, dim, (max(1, dim // 32),), generator=g, device="cuda")] = 4.0
    step = max(1, (1 << 25) // (heads * page * dim))
    for n in range(layers):
        for i in range(0, pages + 1, step):
            m = min(step, pages + 1 - i)
            x = (_randn(g, m, heads, page, dim) * ch * torch.exp2(_randn(g, m, 1, 1, 1))).to(torch.bfloat16).float()
            e = _block_exp(x.abs().amax(dim=(2, 3)))
            exps[n, i:i + m] = e.to(torch.int8)
            codes[n, i:i + m] = _codes(x, e)
    return codes, exps


def _caches(s, g, layers, pages, heads, page, dim):
    s["k"], s["k_exp"] = _fill(g, layers, pages, heads, page, dim)
    s["v"], s["v_exp"] = _fill(g, layers, pages, heads, page, dim)
    s["pages"] = pages


def _prepare_beam(case, g, s):
    B, K, V = case["B"], case["beams"], case["V"]
    x = _randn(g, B, K, V)
    spike = torch.randint(0, V, (B, K, 3), generator=g, device="cuda")
    x.scatter_add_(2, spike, 4 + 8 * torch.rand(B, K, 3, generator=g, device="cuda"))
    s["logits"] = x.to(torch.bfloat16)
    s["scores"] = -20 + 2 * _randn(g, B, K)
    s["done"] = s["weights"] = None
    if case["ends"]:
        s["done"] = (torch.rand(B, K, generator=g, device="cuda") < 0.15).to(torch.int32)
        length = torch.randint(5, 60, (B, K), generator=g, device="cuda")
        s["weights"] = (6.0 / (5.0 + length.float())) ** 0.6


def _prepare_fork(case, seed, g, s):
    """Tables as a beam step finds them: the prompt's full pages shared, the rest each beam's own."""
    NG, per, P = case["groups"], case["per"], case["page"]
    rng = np.random.default_rng([13, int(seed)])
    sizes = np.random.default_rng([17, NG, per, case["prompt"], case["made"], P])  # lengths go by the case alone
    prompt = np.maximum(1, [case["prompt"]] + [int(sizes.integers(max(1, case["prompt"] // 2), case["prompt"] + 1)) for _ in range(NG - 1)])
    made = np.array([case["made"]] + [int(sizes.integers(1, case["made"] + 1)) for _ in range(NG - 1)])
    length = prompt + made
    shared, all_of = prompt // P, -(-length // P)
    used = int(sum(shared) + per * sum(all_of - shared))
    s["n_pages"] = used + 2 * NG * per + 5
    perm, at = rng.permutation(s["n_pages"]).astype(np.int32), 0
    table = np.zeros((NG * per, int(max(all_of)) + 1), np.int32)
    for i in range(NG):
        table[i * per:(i + 1) * per, :shared[i]] = perm[at:at + shared[i]]
        at += shared[i]
        for b in range(i * per, (i + 1) * per):
            own_n = all_of[i] - shared[i]
            table[b, shared[i]:all_of[i]] = perm[at:at + own_n]
            at += own_n
    refs = np.zeros(s["n_pages"], np.int32)
    for b in range(NG * per):
        np.add.at(refs, table[b, :all_of[b // per]], 1)
    for i in range(0, NG, 2):  # every other prompt is also kept for later requests
        refs[table[i * per, :shared[i]]] += 1
    room = np.repeat(length, per)
    parent = np.concatenate([i * per + np.sort(rng.integers(0, per, per)) for i in range(NG)])
    s.update(table=_ints(table), room=_ints(room), parent=_ints(parent), keep=_ints(room), need=_ints(room + 1), refs=_ints(refs))
    _caches(s, g, case["layers"], s["n_pages"], case["heads"], P, case["dim"])


def _prepare_compact(case, seed, g, s):
    """Each sequence's last nodes + 1 positions: the token before the tree, then its nodes."""
    B, T, P = case["B"], case["nodes"], case["page"]
    rng = np.random.default_rng([19, int(seed)])
    sizes = np.random.default_rng([23, B, T, case["kv"], P])
    kv = [case["kv"]] + [int(sizes.integers(max(T + 1, case["kv"] // 2), case["kv"] + 1)) for _ in range(B - 1)]
    need = [-(-n // P) for n in kv]
    perm, at = rng.permutation(sum(need)).astype(np.int32), 0
    table = np.zeros((B, max(need)), np.int32)
    for b in range(B):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    nodes, count = np.full((B, T), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        count[b] = min(T, rng.geometric(0.2) - 1)
        nodes[b, :count[b]] = np.sort(rng.choice(T, count[b], replace=False))
    s.update(cu=_ints(np.arange(B + 1) * (T + 1)), kv=_ints(kv), table=_ints(table), nodes=_ints(nodes), count=_ints(count),
             most=T + 1, T=B * (T + 1))
    _caches(s, g, case["layers"], sum(need), case["heads"], P, case["dim"])


def _prepare_shared(case, seed, g, s):
    NG, per, P, Hk, Hq, D = (case[n] for n in ("groups", "per", "page", "hk", "hq", "dim"))
    rng = np.random.default_rng([29, int(seed)])
    sizes = np.random.default_rng([31, NG, per, case["tok"], case["prefix"], case["suffix"], P, D])
    members = [per] + [int(sizes.integers(max(1, per // 2), per + 1)) if case["ragged"] else per for _ in range(NG - 1)]
    prefix = [case["prefix"]] + [int(sizes.integers(max(1, case["prefix"] // 2), case["prefix"] + 1)) for _ in range(NG - 1)]
    tok, kv, group, table, at, rows = [], [], [], [], 0, []
    for i in range(NG):
        for m in range(members[i]):
            t = case["tok"] if not case["ragged"] or (i, m) == (0, 0) else int(sizes.integers(1, case["tok"] + 1))
            own_n = case["suffix"] if (i, m) == (0, 0) else int(sizes.integers(max(t, case["suffix"] // 4), max(t, case["suffix"]) + 1))
            tok.append(t)
            kv.append(prefix[i] + own_n)
            group.append(i)
    width = max(-(-n // P) for n in kv)
    table = np.zeros((len(kv), width), np.int32)
    for b, n in enumerate(kv):
        i, full = group[b], prefix[group[b]] // P  # full pages of the prefix are shared
        if b == 0 or group[b - 1] != i:
            head = np.arange(at, at + full)
            at += full
        table[b, :full] = head
        mine = -(-n // P) - full
        table[b, full:full + mine] = np.arange(at, at + mine)
        at += mine
    perm = rng.permutation(at).astype(np.int32)
    _caches(s, g, 1, at, Hk, P, D)
    table = perm[table]
    # the prefix's last tokens lie in a page of each sequence's own: all of them copies of the first one's
    src, dst, cut = [], [], []
    for b in range(len(kv)):
        lead, full = group.index(group[b]), prefix[group[b]] // P
        if b != lead and prefix[group[b]] % P:
            src.append(table[lead, full])
            dst.append(table[b, full])
            cut.append(prefix[group[b]] % P)
    if src:
        src, dst = _ints(src).long(), _ints(dst).long()
        old = (torch.arange(P, device="cuda") < _ints(cut)[:, None])[:, None, :, None]
        for side in "kv":
            s[side][0, dst] = torch.where(old, s[side][0, src], s[side][0, dst])
            s[side + "_exp"][0, dst] = s[side + "_exp"][0, src]
    cu = np.concatenate([[0], np.cumsum(tok)])
    s.update(table=_ints(table), kv=_ints(kv), cu=_ints(cu), T=int(cu[-1]), most=max(tok), B=len(kv), prefix=_ints(prefix),
             groups=_ints(np.concatenate([[0], np.cumsum(members)])), per=max(members),
             group_most=max(sum(t for t, j in zip(tok, group) if j == i) for i in range(NG)), prefix_most=max(prefix),
             suffix_most=max(n - prefix[i] for n, i in zip(kv, group)))
    q = _randn(g, s["T"], Hq, D)
    q[..., torch.randint(0, D, (max(1, D // 32),), generator=g, device="cuda")] *= 4.0
    s["q"] = q.to(torch.bfloat16)


def prepare(case, seed):
    g, s = _gen(seed), {"case": case}
    if case["op"] == "beam":
        _prepare_beam(case, g, s)
    elif case["op"] == "fork":
        _prepare_fork(case, seed, g, s)
    elif case["op"] == "compact":
        _prepare_compact(case, seed, g, s)
    else:
        _prepare_shared(case, seed, g, s)
    return s


def work(case):
    if case["op"] == "beam":
        n = case["B"] * case["beams"] * case["V"]
        return {"bytes": 2 * n + case["B"] * (12 * case["beams"] + 12 * case["n"]), "flops": 4 * n}
    if case["op"] == "fork":  # tables and counts in and out, about half the rows' last page (half full) in and out
        rows = case["groups"] * case["per"]
        entries = rows * ((0.75 * case["prompt"] + case["made"] / 2) / case["page"] + 1)
        token = 2 * case["layers"] * case["heads"] * case["dim"]
        return {"bytes": 16 * entries + rows * 0.4 * case["page"] / 2 * token * 2, "flops": 0}
    token = 2 * case.get("layers", 1) * case.get("heads", 1) * case["dim"]
    if case["op"] == "compact":  # the path's codes in and out
        path = min(case["nodes"], 4)
        return {"bytes": case["B"] * path * token * 2, "flops": case["B"] * path * token * 2}
    NG, D, hq, hk = case["groups"], case["dim"], case["hq"], case["hk"]
    mean = lambda most, least: (most + (NG - 1) * (most + least) / 2) / NG  # noqa: E731
    per = mean(case["per"], max(1, case["per"] // 2)) if case["ragged"] else case["per"]
    tok = (case["tok"] + 1) / 2 if case["ragged"] else case["tok"]
    prefix, suffix = mean(case["prefix"], case["prefix"] / 2), max(tok, 0.625 * case["suffix"])
    T = NG * per * tok
    return {"bytes": 2 * hk * D * (NG * prefix + NG * per * suffix) + 4 * T * hq * D,
            "flops": 4 * T * hq * D * (prefix + max(suffix - tok / 2, suffix / 2))}


# ---------------------------------------------------------------------------------------- the plain form

def _beam(s):
    c, x = s["case"], s["logits"]
    B, K, V = x.shape
    n = c["n"]
    bits = x.view(torch.int16).to(torch.int64) & 0xFFFF
    bits = torch.where(bits == 0x8000, torch.zeros_like(bits), bits)                 # -0 is 0
    order = torch.where(bits >= 0x8000, 0xFFFF - bits, bits + 0x8000)                # as the logits are ordered
    key = order * (1 << 24) + ((1 << 24) - 1 - torch.arange(V, device="cuda"))       # equal logits: the lowest token first
    top = torch.topk(key, min(n, V), dim=2, sorted=True).values
    tok = (1 << 24) - 1 - (top & ((1 << 24) - 1))
    z = x.double()
    m = z.amax(2, keepdim=True)
    lse = m + torch.log(torch.exp(z - m).sum(2, keepdim=True))
    S = s["scores"].double()[..., None] + (torch.gather(z, 2, tok) - lse)
    if s["done"] is not None:  # a finished beam stays as it is: one candidate
        done = s["done"][..., None] != 0
        first = torch.arange(S.shape[2], device="cuda") == 0
        S = torch.where(done, torch.where(first, s["scores"].double()[..., None], -math.inf), S)
        tok = torch.where(done, torch.full_like(tok, 2), tok)
    rank = S if s["weights"] is None else S * s["weights"].double()[..., None]
    rank, at = torch.sort(rank.reshape(B, -1), dim=1, descending=True, stable=True)
    at, real = at[:, :n], rank[:, :n] > -math.inf
    parent = torch.arange(B, device="cuda")[:, None] * K + at // S.shape[2]
    return {"parent": torch.where(real, parent, -1).to(torch.int32),
            "tok": torch.where(real, torch.gather(tok.reshape(B, -1), 1, at), -1).to(torch.int32),
            "score": torch.gather(S.reshape(B, -1), 1, at).float()}


def _fork(s):
    c = s["case"]
    P, R, W, N = c["page"], s["table"].shape[0], s["table"].shape[1], s["n_pages"]
    table, room, parent, keep, need = (s[n].long() for n in ("table", "room", "parent", "keep", "need"))
    j = torch.arange(W, device="cuda")
    had = j < ((room + P - 1) // P)[:, None]
    kept, got = (keep + P - 1) // P, (need + P - 1) // P
    new = table[parent]
    stays = j < kept[:, None]
    refs = s["refs"].long()
    refs = refs.scatter_add(0, new.reshape(-1), stays.reshape(-1).long()).scatter_add(0, table.reshape(-1), -had.reshape(-1).long())
    # the page that a row goes on writing in
    writes = (keep % P != 0) & (need > keep)
    last = torch.gather(new, 1, (keep // P).clamp(max=W - 1)[:, None])[:, 0]
    at = torch.where(writes, last, N)
    writers = torch.zeros(N + 1, dtype=torch.int64, device="cuda").scatter_add_(0, at, torch.ones_like(at))
    row = torch.arange(R, device="cuda")
    lowest = torch.full((N + 1,), R, dtype=torch.int64, device="cuda").scatter_reduce_(0, at, row, "amin")
    copies = writes & ((refs[last] != writers[last]) | (lowest[last] != row))
    # free pages, lowest first, to the rows in order
    take = got - kept + copies.long()
    start = take.cumsum(0) - take
    free = refs == 0
    nth = torch.where(free, free.long().cumsum(0) - 1, N)
    ids = torch.zeros(N + 1, dtype=torch.int64, device="cuda").scatter_(0, nth, torch.arange(N, device="cuda"))
    first = kept - copies.long()
    fresh = (j >= first[:, None]) & (j < got[:, None])
    pick = ids[(start[:, None] + j - first[:, None]).clamp(0, N)]
    new = torch.where(fresh, pick, torch.where(j < got[:, None], new, 0))
    refs = refs.scatter_add(0, last, -copies.long()).scatter_add(0, torch.where(fresh, pick, 0).reshape(-1), fresh.reshape(-1).long())
    dst = torch.gather(new, 1, (keep // P).clamp(max=W - 1)[:, None])[:, 0]
    size = torch.where(copies, keep % P, 0)
    # the copies themselves, in every layer
    to = torch.where(copies, dst, N)
    old = (torch.arange(P, device="cuda") < size[:, None])[None, :, None, :, None]
    for side in "kv":
        s[side][:, to] = torch.where(old, s[side][:, last], s[side][:, to])
        s[side + "_exp"][:, to] = s[side + "_exp"][:, last]
    i32 = lambda t: t.to(torch.int32)  # noqa: E731
    return {"table": i32(new), "refs": i32(refs), "src": i32(torch.where(copies, last, -1)), "dst": i32(torch.where(copies, dst, -1)),
            "len": i32(size), "left": i32(free.sum() - take.sum())}


def _compact(s):
    c = s["case"]
    P, T = c["page"], c["nodes"]
    kv, count, nodes = s["kv"].long(), s["count"].long(), s["nodes"].long()
    first = kv - T                                                   # where node 0 lies, and the path begins
    page0, W = first // P, (T + P - 2) // P + 1
    j = page0[:, None] + torch.arange(W, device="cuda")
    in_table = j < s["table"].shape[1]
    page = torch.where(in_table & (j * P < kv[:, None]), torch.gather(s["table"].long(), 1, j.clamp(max=s["table"].shape[1] - 1)), s["pages"])
    pos = page0[:, None] * P + torch.arange(W * P, device="cuda")   # [B, W P]
    i = pos - first[:, None]
    moved = (i >= 0) & (i < count[:, None])
    node = torch.gather(nodes, 1, i.clamp(0, T - 1))
    source = torch.where(moved, node + (first - page0 * P)[:, None], torch.arange(W * P, device="cuda"))
    for side in "kv":
        codes, exps = s[side], s[side + "_exp"]
        L, _, H, _, D = codes.shape
        old, e_old = codes[:, page], exps[:, page].int()             # [L, B, W, H, P, D], [L, B, W, H]
        x = _values(old, e_old).permute(0, 1, 3, 2, 4, 5).reshape(L, -1, H, W * P, D)
        x = torch.gather(x, 3, source[None, :, None, :, None].expand(L, -1, H, -1, D)).view(L, -1, H, W, P, D).permute(0, 1, 3, 2, 4, 5)
        put = moved.view(-1, W, P)
        amax = (x.abs().amax(5) * put[None, :, :, None, :]).amax(4)
        begun = put[:, :, 0][None, :, :, None]                      # what else lies in such a page means nothing any more
        e_new = torch.where(begun, _block_exp(amax), torch.maximum(e_old, _block_exp(amax)))
        e_new = torch.where(put.any(2)[None, :, :, None], e_new, e_old)
        keep = (~put)[None, :, :, None, :, None] & (begun | (e_new == e_old))[..., None, None]
        codes[:, page] = torch.where(keep, old, _codes(x, e_new))
        exps[:, page] = e_new.to(torch.int8)


def _rows_of(s):
    """Of each token: its sequence, and its index among the sequence's new tokens."""
    cu = s["cu"].long()
    t = torch.arange(s["T"], device="cuda")
    b = (t[:, None] >= cu[None, 1:]).sum(1)
    return b, t - cu[b]


def _part(q, K, V, see, scale):
    """Softmax sums of q [N, H, R, D] over K, V [N, H, L, D] where see [N, 1, R, L]: (sum of p v, sum of p, maximum)."""
    S = (q @ K.transpose(2, 3)) * scale
    S = S.masked_fill(~see, -math.inf)
    m = S.amax(-1, keepdim=True)
    p = torch.exp(S - torch.where(m == -math.inf, 0.0, m))
    return p @ V, p.sum(-1, keepdim=True), m


def _shared(s):
    c = s["case"]
    P, Hk, D, G = c["page"], c["hk"], c["dim"], c["hq"] // c["hk"]
    B, most, per, NG = s["B"], s["most"], s["per"], s["groups"].numel() - 1
    cu, kv, prefix, first = s["cu"].long(), s["kv"].long(), s["prefix"].long(), s["groups"].long()
    scale = 1.0 / math.sqrt(D)
    seq = torch.arange(B, device="cuda")
    of = (seq[:, None] >= first[None, 1:]).sum(1)                     # the group of each sequence

    def values(side, page):                                           # pages [N, W] -> [N, Hk, W P, D]
        x = _values(s[side][0, page], s[side + "_exp"][0, page])
        return x.permute(0, 2, 1, 3, 4).reshape(page.shape[0], Hk, -1, D)

    row = (cu[:-1, None] + torch.arange(most, device="cuda")).clamp(max=s["T"] - 1)
    Q = s["q"].float()[row].view(B, most, Hk, G, D).permute(0, 2, 1, 3, 4)   # [B, Hk, most, G, D]
    # the prefix: all rows of a group at once
    member = (first[:-1, None] + torch.arange(per, device="cuda")).clamp(max=B - 1)
    Wp = -(-s["prefix_most"] // P)
    page = s["table"].long()[first[:-1], :Wp]
    q = Q[member].permute(0, 2, 1, 3, 4, 5).reshape(NG, Hk, per * most * G, D)
    see = (torch.arange(Wp * P, device="cuda") < prefix[:, None])[:, None, None, :]
    op, lp, mp = _part(q, values("k", page), values("v", page), see, scale)
    back = lambda t: t.view(NG, Hk, per, most * G, -1).permute(0, 2, 1, 3, 4)[of, seq - first[of]]  # noqa: E731
    op, lp, mp = back(op), back(lp), back(mp)                        # [B, Hk, most G, ...]
    # what each sequence has alone
    p0 = prefix[of] // P
    Ws = -(-s["suffix_most"] // P) + 1
    page = torch.gather(s["table"].long(), 1, (p0[:, None] + torch.arange(Ws, device="cuda")).clamp(max=s["table"].shape[1] - 1))
    j = p0[:, None] * P + torch.arange(Ws * P, device="cuda")
    at = (kv - (cu[1:] - cu[:-1]))[:, None] + torch.arange(most, device="cuda")
    see = (j[:, None] >= prefix[of][:, None, None]) & (j[:, None] <= at[..., None]) & (j[:, None] < kv[:, None, None])
    see = see[:, None, :, None].expand(-1, -1, -1, G, -1).reshape(B, 1, most * G, -1)
    os_, ls, ms = _part(Q.reshape(B, Hk, most * G, D), values("k", page), values("v", page), see, scale)
    m = torch.maximum(mp, ms)
    fp, fs = torch.exp(mp - m), torch.exp(ms - m)
    l = lp * fp + ls * fs
    O, lse = (op * fp + os_ * fs) / l, m + torch.log(l)
    b, i = _rows_of(s)
    out = O.view(B, Hk, most, G, D).permute(0, 2, 1, 3, 4)[b, i].reshape(s["T"], Hk * G, D)
    lse = lse.view(B, Hk, most, G).permute(0, 2, 1, 3)[b, i].reshape(s["T"], Hk * G)
    return {"out": out.to(torch.bfloat16), "lse": lse}


# ---------------------------------------------------------------------------------------- the library's calls

def _layers(s, lib):
    caches = [lib.KVCache(s["k"][n, :s["pages"]], s["v"][n, :s["pages"]], s["k_exp"][n, :s["pages"]], s["v_exp"][n, :s["pages"]])
              for n in range(s["k"].shape[0])]
    return lib.KVLayers(caches)


def _handles(s):
    """What a user's program makes once: the cache and batch descriptions, workspaces and output buffers."""
    from quantized_speculative_decoding_qspec_gb300 import qspec as lib
    c, h = s["case"], {"lib": lib}
    new = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device="cuda")  # noqa: E731
    if c["op"] == "beam":
        h.update(parent=new(c["B"], c["n"]), tok=new(c["B"], c["n"]), score=torch.empty(c["B"], c["n"], device="cuda"),
                 ws=lib.new_beam_workspace(c["B"], c["beams"], c["V"], c["n"]))
    elif c["op"] == "fork":
        R = s["table"].shape[0]
        h.update(layers=_layers(s, lib), table=torch.zeros_like(s["table"]), refs=torch.empty_like(s["refs"]), src=new(R), dst=new(R),
                 len=new(R), left=new(1))
    elif c["op"] == "compact":
        h.update(layers=_layers(s, lib), batch=lib.KVBatch(s["cu"], s["kv"], s["table"], s["most"]))
    else:
        h.update(cache=_layers(s, lib).caches[0], batch=lib.KVBatch(s["cu"], s["kv"], s["table"], s["most"]),
                 prefixes=lib.KVPrefixes(s["groups"], s["prefix"], s["group_most"]), out=torch.empty_like(s["q"]),
                 lse=torch.empty(s["T"], c["hq"], dtype=torch.float32, device="cuda"), ws=lib.new_kv_attention_workspace())
    return h


def _contents(s):
    """The caches as the values that their codes stand for."""
    n = s["pages"]
    return {"k": s["k"][:, :n].view(torch.float8_e4m3fn), "v": s["v"][:, :n].view(torch.float8_e4m3fn),
            "k_exp": s["k_exp"][:, :n], "v_exp": s["v_exp"][:, :n]}


def run(s):
    c = s["case"]
    if own and "handles" not in s:
        s["handles"] = _handles(s)
    h = s.get("handles") if own else None
    if c["op"] == "beam":
        if not own:
            return _beam(s)
        h["lib"].qspec_beam_select(s["logits"], s["scores"], h["parent"], h["tok"], h["score"], h["ws"], done=s["done"], end_tok=2,
                                   weights=s["weights"])
        return {"parent": h["parent"], "tok": h["tok"], "score": h["score"]}
    if c["op"] == "fork":
        if not own:
            return dict(_fork(s), **_contents(s))
        lib = h["lib"]
        lib.qspec_kv_pages(s["table"], s["room"], s["keep"], s["need"], s["refs"], c["page"], h["table"], h["refs"], h["src"], h["dst"],
                           h["len"], h["left"], parent=s["parent"])
        lib.qspec_kv_copy_pages(h["layers"], h["src"], h["dst"], lengths=h["len"])
        return dict({n: h[n] for n in ("table", "refs", "src", "dst", "len")}, left=h["left"][0], **_contents(s))
    if c["op"] == "compact":
        if own:
            h["lib"].qspec_kv_compact(h["layers"], h["batch"], s["nodes"], s["count"], first=1)
        else:
            _compact(s)
        return _contents(s)
    if not own:
        return _shared(s)
    h["lib"].qspec_kv_attention_shared(h["cache"], h["batch"], h["prefixes"], s["q"], h["out"], h["ws"], lse=h["lse"])
    return {"out": h["out"], "lse": h["lse"]}


# ---------------------------------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None  # whole numbers, and codes that are what the rounding gives
    s = prepare(case, seed)
    if case["op"] == "beam":
        B, K, V = s["logits"].shape
        score = torch.full((B, case["n"]), -math.inf, dtype=torch.float64, device="cuda")
        for b in range(B):
            best = []
            for k in range(K):
                start = float(s["scores"][b, k])
                w = 1.0 if s["weights"] is None else float(s["weights"][b, k])
                if s["done"] is not None and int(s["done"][b, k]):
                    best.append((start * w, start))
                    continue
                lp = torch.log_softmax(s["logits"][b, k].double(), 0) + start
                best += [(float(v) * w, float(v)) for v in torch.topk(lp, min(case["n"], V)).values]
            best.sort(key=lambda t: -t[0])
            for n, (_, v) in enumerate(best[:case["n"]]):
                score[b, n] = v
        return {"parent": None, "tok": None, "score": score}
    P, Hk, G, D = case["page"], case["hk"], case["hq"] // case["hk"], case["dim"]
    cu, kv = s["cu"].tolist(), s["kv"].tolist()
    out = torch.zeros(s["T"], Hk * G, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["T"], Hk * G, dtype=torch.float64, device="cuda")
    for b in range(s["B"]):
        ids, n = s["table"][b, :-(-kv[b] // P)].long(), cu[b + 1] - cu[b]
        K, V = ((s[a][0, ids].view(torch.float8_e4m3fn).double() * 2.0 ** s[a + "_exp"][0, ids].double()[..., None, None])
                .transpose(0, 1).reshape(Hk, -1, D)[:, :kv[b]] for a in "kv")
        i = torch.arange(n, device="cuda")[:, None] + kv[b] - n
        off = torch.where(torch.arange(kv[b], device="cuda") <= i, 0.0, -math.inf).double()
        Q = s["q"][cu[b]:cu[b + 1]].double().view(n, Hk, G, D)
        S = torch.einsum("thgd,hjd->htgj", Q, K) / D ** 0.5 + off[None, :, None]
        lse[cu[b]:cu[b + 1]] = torch.logsumexp(S, -1).permute(1, 0, 2).reshape(n, -1)
        out[cu[b]:cu[b + 1]] = torch.einsum("htgj,hjd->thgd", torch.softmax(S, -1), V).reshape(n, -1, D)
    return {"out": out, "lse": lse}
