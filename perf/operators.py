"""What a speculative decode step needs around the 4-bit linears, as measured cases.

Four operators, one pass each:

* rotary    -- rotary positions of a [tokens, heads, dim] tensor (half or interleaved pairs, part of
               the head, frequencies scaled for long contexts, forward or inverse);
* append    -- the step's new keys and values into a paged cache of e4m3 codes with one power-of-two
               scale per page and head, keys (and queries) rotated on the way;
* attention -- causal attention of the step's queries over that cache (one token, the gamma + 1
               positions of a verify pass, the nodes of a candidate tree, a chunk of a prompt);
* logits    -- repetition, frequency and presence penalties, biases and a grammar mask on the
               logits of the gamma + 1 positions, where position i counts the draft tokens before it.

``own`` False: the plain form, elementary torch operations in fp32 (fp64 for the angles).
``own`` True: the calls a user makes of the library.  Head counts, page sizes, vocabularies and
draft lengths are those of the decode shapes that the benchmark and the tests use (4096-wide layers
with 32 heads and 8 key heads of 128, 8192-wide ones with 64 and 8; vocabularies of 32000, 128256
and 152064; draft lengths 1 to 7), or generic.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
EXP_MIN, EXP_MAX = -40, 40


# ---------------------------------------------------------------------------------------- cases

def listed():
    att = {"op": "attention", "dim": 128, "page": 64, "window": 0, "tree": False}
    return [
        # one token of one sequence through 32 query heads: pure latency
        {"name": "rotary_token", "op": "rotary", "T": 1, "heads": 32, "dim": 128, "rot": 128, "inter": False,
         "scaling": "none", "factor": 1.0, "far": 8192, "inverse": False, "pad": 0},
        # a prompt's queries and keys as slices of one projection output (strided rows), part of the
        # head, interleaved pairs, positions beyond the trained range, the inverse direction
        {"name": "rotary_prompt", "op": "rotary", "T": 8192, "heads": 40, "dim": 128, "rot": 96, "inter": True,
         "scaling": "yarn", "factor": 16.0, "far": 1 << 20, "inverse": True, "pad": 1024},
        # a verify pass of 16 sequences: 4 new tokens each, queries rotated in the same call
        {"name": "append_verify", "op": "append", "B": 16, "tok": 4, "ragged": False, "kv": 4096, "hq": 32, "hk": 8,
         "dim": 128, "page": 64, "inter": False, "scaling": "bands", "factor": 8.0},
        # prompts of different lengths written at once
        {"name": "append_prompt", "op": "append", "B": 4, "tok": 4096, "ragged": True, "kv": 8192, "hq": 32, "hk": 8,
         "dim": 128, "page": 64, "inter": False, "scaling": "bands", "factor": 8.0},
        # a short conversation, one token: the smallest attention
        dict(att, name="att_token", B=1, tok=1, ragged=False, kv=517, hq=32, hk=8),
        # a verify pass of 16 sequences of different lengths, draft length 3
        dict(att, name="att_verify", B=16, tok=4, ragged=False, kv=8192, hq=32, hk=8),
        # a large decode batch, one token each, 8 query heads to a key head
        dict(att, name="att_batch", B=64, tok=1, ragged=False, kv=6001, hq=64, hk=8),
        # one sequence with a long context, draft length 3
        dict(att, name="att_long", B=1, tok=4, ragged=False, kv=131072, hq=32, hk=8),
        # candidate trees of up to 31 nodes, heads of 64, small pages
        dict(att, name="att_tree", B=8, tok=31, ragged=True, kv=2049, hq=16, hk=16, dim=64, page=16, tree=True),
        # the second half of a prompt, in one chunk
        dict(att, name="att_prompt", B=1, tok=4096, ragged=False, kv=8192, hq=32, hk=8),
        # one sequence's verify rows, penalties and a few biases
        {"name": "logits_one", "op": "logits", "B": 1, "gamma": 3, "V": 128256, "hist": 1500, "bias": 40, "mask": False},
        # a batch's verify rows, long histories, grammar masks
        {"name": "logits_batch", "op": "logits", "B": 64, "gamma": 7, "V": 152064, "hist": 8192, "bias": 300, "mask": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "attention", "attention", "attention", "logits"])
    scaling = rng.choice(["none", "linear", "base", "bands", "yarn"])
    factor = 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 16.0])
    if op == "rotary":
        dim = rng.choice([64, 128])
        return {"op": op, "T": _log(rng, 1, 8192), "heads": rng.choice([1, 8, 16, 32, 40]), "dim": dim,
                "rot": rng.choice([dim, dim // 2, dim * 3 // 4]), "inter": rng.random() < 0.5, "scaling": scaling,
                "factor": factor, "far": _log(rng, 4096, 1 << 20), "inverse": rng.random() < 0.3,
                "pad": rng.choice([0, 8, 1024])}
    if op == "append":
        B = _log(rng, 1, 64)
        return {"op": op, "B": B, "tok": _log(rng, 1, max(1, 16384 // B)), "ragged": rng.random() < 0.5,
                "kv": _log(rng, 16, max(16, 32768 // B)), "hq": rng.choice([32, 64]), "hk": 8, "dim": rng.choice([64, 128]),
                "page": rng.choice([16, 32, 64, 128]), "inter": rng.random() < 0.5, "scaling": scaling, "factor": factor}
    if op == "logits":
        B = _log(rng, 1, 64)
        return {"op": op, "B": B, "gamma": rng.choice([1, 3, 5, 7]), "V": rng.choice([32000, 50001, 128256, 152064]),
                "hist": _log(rng, 1, 8192), "bias": rng.choice([0, 7, 300]), "mask": rng.random() < 0.5}
    hk, g = rng.choice([(8, 4), (8, 8), (8, 1), (2, 7), (1, 8)])
    kind = rng.choice(["token", "verify", "tree", "chunk"])
    tok = {"token": 1, "verify": rng.randint(2, 8), "tree": rng.randint(2, 64), "chunk": _log(rng, 16, 2048)}[kind]
    B = _log(rng, 1, 4 if kind == "chunk" else 64)
    kv = _log(rng, 16, 8192 if kind == "chunk" else max(64, 262144 // B))
    kv = min(kv, (1 << 30) // (B * tok * hk * g))
    return {"op": op, "B": B, "tok": tok, "ragged": rng.random() < 0.5, "kv": max(kv, tok), "hq": hk * g, "hk": hk,
            "dim": rng.choice([64, 128, 128]), "page": rng.choice([16, 32, 64, 128]),
            "window": rng.choice([0, 0, 0, 1024]) if kind != "tree" else 0, "tree": kind == "tree"}


# ---------------------------------------------------------------------------------------- inputs

ROPE = {"base": 500000.0, "orig": 8192, "low": 1.0, "high": 4.0, "fast": 32.0, "slow": 1.0}


def _lengths(rng, B, most, ragged):
    """The longest first, the others anywhere below (at least one)."""
    return [most] + [int(rng.integers(1, most + 1)) if ragged else most for _ in range(B - 1)]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _heads(g, T, H, D, channel):
    """Activations of one projection: unit normal, a few channels larger, as keys and queries have them."""
    return (_randn(g, T, H, D) * channel).to(torch.bfloat16)


def _channels(g, H, D):
    c = torch.ones(H, D, device="cuda")
    c[:, torch.randint(0, D, (max(1, D // 32),), generator=g, device="cuda")] = 4.0
    return c


def _block_exp(amax):
    """The smallest e with amax <= 448 * 2^e, within the limits; amax fp32 with a bf16 value."""
    m, k = torch.frexp(amax)                       # amax = m * 2^k, m in [0.5, 1)
    e = torch.where(m > 0.875, k - 8, k - 9)       # 448 = 0.875 * 2^9
    return torch.where(amax > 0, e, torch.full_like(e, EXP_MIN)).clamp(EXP_MIN, EXP_MAX)


def _fill_cache(g, pages, heads, page, dim):
    """A cache as earlier steps left it: every page quantised from normal values, in slices of pages."""
    codes = torch.empty(pages, heads, page, dim, dtype=torch.uint8, device="cuda")
    exps = torch.empty(pages, heads, dtype=torch.int8, device="cuda")
    step = max(1, (1 << 25) // (heads * page * dim))
    ch = _channels(g, heads, dim)[None, :, None, :]
    for i in range(0, pages, step):
        n = min(step, pages - i)
        x = (_randn(g, n, heads, page, dim) * ch * torch.exp2(_randn(g, n, 1, 1, 1))).to(torch.bfloat16).float()
        e = _block_exp(x.abs().amax(dim=(2, 3)))
        exps[i:i + n] = e.to(torch.int8)
        codes[i:i + n] = (x * torch.exp2(-e.float())[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, exps


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _page_table(g, case, kv):
    B, P = case["B"], case["page"]
    need = [-(-n // P) for n in kv]
    width = max(need)
    perm = torch.randperm(sum(need), generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, sum(need)


def prepare(case, seed):
    g, rng = _gen(seed), np.random.default_rng([7, int(seed)])
    s = {"case": case}
    if case["op"] == "rotary":
        T, H, D = case["T"], case["heads"], case["dim"]
        buf = torch.empty(T, H * D + case["pad"], dtype=torch.bfloat16, device="cuda")
        x = buf[:, :H * D].view(T, H, D)
        x.copy_(_heads(g, T, H, D, _channels(g, H, D)))
        first = int(rng.integers(0, max(1, case["far"] - T)))
        s.update(x=x, pos=torch.arange(first, first + T, dtype=torch.int32, device="cuda"))
        return s
    if case["op"] == "logits":
        B, G1, V = case["B"], case["gamma"] + 1, case["V"]
        x = _randn(g, B, G1, V)
        spike = torch.randint(0, V, (B, G1, 1), generator=g, device="cuda")
        x.scatter_add_(2, spike, 4 + 8 * torch.rand(B, G1, 1, generator=g, device="cuda"))
        hist = (torch.rand(B, case["hist"], generator=g, device="cuda") ** 6 * V).to(torch.int32).clamp_(0, V - 1)
        hl = _lengths(rng, B, case["hist"], True)
        s.update(logits=x.to(torch.bfloat16), draft=spike[:, :G1 - 1, 0].to(torch.int32).contiguous(),
                 hist=hist, hist_len=_ints(hl), prompt_len=_ints([int(rng.integers(0, n + 1)) for n in hl]),
                 pen=torch.tensor(np.stack([rng.uniform(1.0, 1.3, B), rng.uniform(0, 0.5, B), rng.uniform(0, 0.5, B)], 1),
                                  dtype=torch.float32, device="cuda"),
                 bias_id=None, bias=None, mask=None)
        if case["bias"]:
            ids = torch.stack([torch.randperm(V, generator=g, device="cuda")[:case["bias"]] for _ in range(B)]).to(torch.int32)
            ids[:, case["bias"] - case["bias"] // 8:] = -1  # lists of different lengths end in -1
            s.update(bias_id=ids, bias=_randn(g, B, case["bias"]) * 3)
        if case["mask"]:
            s["mask"] = torch.randint(-2 ** 31, 2 ** 31, (B, G1, (V + 31) // 32), generator=g, device="cuda").to(torch.int32)
        return s
    B, P, Hk, Hq, D = case["B"], case["page"], case["hk"], case["hq"], case["dim"]
    # lengths go by the case alone: inputs of another seed have the same shapes
    sizes = np.random.default_rng([11, B, case["tok"], case["kv"], P, D, Hq])
    tok = _lengths(sizes, B, case["tok"], case["ragged"])
    # contexts of a served batch differ: the longest as given, the others a quarter of it and more
    kv = [case["kv"]] + [int(sizes.integers(max(1, case["kv"] // 4), case["kv"] + 1)) for _ in range(B - 1)]
    kv = [max(n, t) for n, t in zip(kv, tok)]
    T = sum(tok)
    table, pages = _page_table(g, case, kv)
    s["k"], s["k_exp"] = _fill_cache(g, pages, Hk, P, D)
    s["v"], s["v_exp"] = _fill_cache(g, pages, Hk, P, D)
    s.update(cu=_ints([0] + list(np.cumsum(tok))), kv=_ints(kv), table=table, most=max(tok), T=T)
    s["q"] = _heads(g, T, Hq, D, _channels(g, Hq, D))
    if case["op"] == "append":
        s["k_new"] = _heads(g, T, Hk, D, _channels(g, Hk, D))
        s["v_new"] = _heads(g, T, Hk, D, _channels(g, Hk, D))
    else:
        s["tree"] = None
        if case["tree"]:  # each node's bits: its ancestors and itself
            rows = []
            for n in tok:
                anc = []
                for j in range(n):
                    p = int(rng.integers(-1, j)) if j else -1
                    anc.append((anc[p] if p >= 0 else 0) | 1 << j)
                rows += anc
            s["tree"] = torch.from_numpy(np.array(rows, dtype=np.uint64).view(np.int64)).cuda()
    return s


def work(case):
    if case["op"] == "rotary":
        n = case["T"] * case["heads"] * case["dim"]
        return {"bytes": 4 * n + 4 * case["T"], "flops": 3 * case["T"] * case["heads"] * case["rot"]}
    if case["op"] == "logits":
        rows = case["B"] * (case["gamma"] + 1)
        return {"bytes": rows * case["V"] * (4.125 if case["mask"] else 4) + case["B"] * (2 * case["hist"] + 8 * case["bias"]),
                "flops": rows * case["V"]}
    B, D, hq, hk = case["B"], case["dim"], case["hq"], case["hk"]
    mean_tok = case["tok"] if not case["ragged"] else (case["tok"] + (B - 1) * (case["tok"] + 1) / 2) / B
    mean_kv = (case["kv"] + (B - 1) * 0.625 * case["kv"]) / B
    T = B * mean_tok
    if case["op"] == "append":  # queries in and out, new keys and values in, their codes out
        return {"bytes": T * D * (4 * hq + 4 * hk + 2 * hk), "flops": T * D * 3 * (hq + hk)}
    see = max(mean_kv - mean_tok / 2, mean_kv / 2)
    kv = mean_kv
    if case["window"]:
        see, kv = min(see, case["window"]), min(kv, case["window"] + mean_tok)
    return {"bytes": 2 * B * kv * hk * D + 4 * T * hq * D, "flops": 4 * T * hq * D * see}


# ---------------------------------------------------------------------------------------- the plain form

def _inv_freq(rot, scaling, factor):
    """Radians per position of each pair (fp64), and the factor on the rotated values."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    base, orig = ROPE["base"], ROPE["orig"]
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    inv = base ** (-2 * i / rot)
    if scaling == "linear":
        return inv / factor, 1.0
    if scaling == "bands":
        turns = orig * inv / (2 * math.pi)
        part = ((turns - ROPE["low"]) / (ROPE["high"] - ROPE["low"])).clamp(0, 1)
        return (1 - part) * inv / factor + part * inv, 1.0
    if scaling == "yarn":
        def edge(beta):
            return rot * math.log(orig / (beta * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(edge(ROPE["fast"])), 0), min(math.ceil(edge(ROPE["slow"])), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return inv / factor * ramp + inv * (1 - ramp), 0.1 * math.log(factor) + 1 if factor > 1 else 1.0
    return inv, 1.0


def _rotate(x, pos, rot, inter, scaling, factor, inverse=False):
    """x [T, H, D] bf16 -> rotated, bf16.  Angles and their cosines in fp64."""
    inv, mult = _inv_freq(rot, scaling, factor)
    ang = pos.double()[:, None] * inv
    cos, sin = (ang.cos() * mult).float()[:, None, :], (ang.sin() * mult).float()[:, None, :]
    if inverse:
        sin = -sin
    y = x.float().clone()
    a, b = (y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()) if inter else (y[..., :rot // 2].clone(), y[..., rot // 2:rot].clone())
    ra, rb = a * cos - b * sin, a * sin + b * cos
    if inter:
        y[..., 0:rot:2], y[..., 1:rot:2] = ra, rb
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = ra, rb
    return y.to(torch.bfloat16)


def _token_places(s):
    """Of each of the T tokens: its sequence, its index in the sequence's new tokens, its cache position."""
    cu = s["cu"].long()
    t = torch.arange(s["T"], device="cuda")
    b = (t[:, None] >= cu[None, 1:]).sum(1)
    i = t - cu[b]
    return b, i, s["kv"].long()[b] - (cu[b + 1] - cu[b]) + i


def _write(codes, exps, new, page_id, slot):
    """Quantises new [T, H, D] (bf16) into their pages; pages that grow are quantised again."""
    n, H, P, D = codes.shape
    x = new.float()
    amax = torch.zeros(n, H, device="cuda").scatter_reduce_(0, page_id[:, None].expand(-1, H), x.abs().amax(2), "amax")
    hit = torch.zeros(n, dtype=torch.bool, device="cuda").index_fill_(0, page_id, True)[:, None]
    first = torch.zeros(n, device="cuda").index_add_(0, page_id, (slot == 0).float())[:, None] > 0  # begun by this call
    old = exps.int()
    e = torch.where(first, _block_exp(amax), torch.maximum(old, _block_exp(amax)))
    e = torch.where(hit, e, old)
    again = codes.view(torch.float8_e4m3fn).float() * torch.exp2((old - e).float())[:, :, None, None]
    again = again.to(torch.float8_e4m3fn).view(torch.uint8)
    codes.copy_(torch.where((~first & (e != old))[:, :, None, None], again, codes))
    exps.copy_(e.to(torch.int8))
    codes[page_id, :, slot] = (x * torch.exp2(-e[page_id].float())[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _append(s):
    c = s["case"]
    b, _, pos = _token_places(s)
    page_id, slot = s["table"][b, pos // c["page"]].long(), pos % c["page"]
    rope = (c["dim"], c["inter"], c["scaling"], c["factor"])
    q = _rotate(s["q"], pos, *rope)
    _write(s["k"], s["k_exp"], _rotate(s["k_new"], pos, *rope), page_id, slot)
    _write(s["v"], s["v_exp"], s["v_new"], page_id, slot)
    return q


def _values(codes, exps, table):
    """The pages of each sequence as fp32 [B, H, length, D]."""
    B, W = table.shape
    _, H, P, D = codes.shape
    x = codes[table.long()].view(torch.float8_e4m3fn).float() * torch.exp2(exps[table.long()].float())[..., None, None]
    return x.permute(0, 2, 1, 3, 4).reshape(B, H, W * P, D)


def _attention(s):
    c = s["case"]
    B, Hk, G, D, most = c["B"], c["hk"], c["hq"] // c["hk"], c["dim"], s["most"]
    K, V = _values(s["k"], s["k_exp"], s["table"]), _values(s["v"], s["v_exp"], s["table"])
    L = K.shape[2]
    cu, kv = s["cu"].long(), s["kv"].long()
    row = cu[:-1, None] + torch.arange(most, device="cuda")
    Q = s["q"].float()[row.clamp(max=s["T"] - 1)].view(B, most, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, most * G, D)
    S = (Q @ K.transpose(2, 3)).view(B, Hk, most, G, L) * (1.0 / math.sqrt(D))
    j = torch.arange(L, device="cuda")
    base = kv - (cu[1:] - cu[:-1])                              # context before the new tokens
    at = base[:, None] + torch.arange(most, device="cuda")      # [B, most]
    if s["tree"] is not None:
        bits = s["tree"][row.clamp(max=s["T"] - 1)][..., None]  # [B, most, 1]
        k = j - base[:, None, None]                             # node of each key
        see = (k < 0) | ((k < 64) & ((bits >> k.clamp(0, 63)) & 1).bool())
        see = see & (j < kv[:, None, None])
    else:
        see = (j <= at[..., None]) & (j < kv[:, None, None])
        if c["window"]:
            see = see & (j > at[..., None] - c["window"])
    see = see[:, None, :, None, :]
    S = S.masked_fill(~see, -math.inf)
    m = S.amax(-1, keepdim=True)
    p = torch.exp(S - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    O = (p.view(B, Hk, most * G, L) @ V).view(B, Hk, most, G, D) / torch.where(l > 0, l, torch.ones_like(l))
    b, i, _ = _token_places(s)
    out = O.permute(0, 2, 1, 3, 4)[b, i].reshape(s["T"], Hk * G, D)
    lse = (m + torch.log(l)).permute(0, 2, 1, 3, 4)[b, i].reshape(s["T"], Hk * G)
    return out.to(torch.bfloat16), lse


def _logits(s):
    x = s["logits"]
    B, G1, V = x.shape
    z = x.float()
    k = torch.arange(s["hist"].shape[1], device="cuda")
    real = k < s["hist_len"][:, None]
    made = real & (k >= s["prompt_len"][:, None])
    ids = s["hist"].long()
    seen = torch.zeros(B, V, device="cuda").scatter_add_(1, ids, real.float())
    cnt = torch.zeros(B, V, device="cuda").scatter_add_(1, ids, made.float())
    # position i has the draft tokens before it in its history
    before = torch.zeros(B, G1, V, device="cuda")
    before[:, 1:].scatter_(2, s["draft"].long()[..., None], 1.0)
    before = before.cumsum(1)
    seen, cnt = (seen[:, None] + before) > 0, cnt[:, None] + before
    rep, freq, pres = (s["pen"][:, n, None, None] for n in range(3))
    z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
    z = z - freq * cnt - pres * (cnt > 0)
    if s["bias_id"] is not None:
        use = s["bias_id"] >= 0
        z = z + torch.zeros(B, V, device="cuda").scatter_add_(1, s["bias_id"].long().clamp(min=0), s["bias"] * use)[:, None]
    if s["mask"] is not None:
        v = torch.arange(V, device="cuda")
        z = z.masked_fill(((s["mask"][..., v // 32] >> (v % 32)) & 1) == 0, -math.inf)
    return z.to(torch.bfloat16)


# ---------------------------------------------------------------------------------------- the library's calls

def _handles(s):
    """What a user's program makes once: the rotary plan, the cache and batch descriptions, the workspace and the output buffers."""
    from quantized_speculative_decoding_qspec_gb300 import qspec as lib
    c, h = s["case"], {"lib": lib}
    if c["op"] in ("rotary", "append"):
        h["rope"] = lib.Rotary(c["rot"] if c["op"] == "rotary" else c["dim"], base=ROPE["base"], interleaved=c["inter"],
                               scaling=c["scaling"], factor=c["factor"], original=ROPE["orig"], low=ROPE["low"],
                               high=ROPE["high"], fast=ROPE["fast"], slow=ROPE["slow"])
    if c["op"] == "rotary":
        h["out"] = torch.empty(s["x"].shape, dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "logits":
        h["out"] = torch.empty_like(s["logits"])
    else:
        h["cache"] = lib.KVCache(s["k"], s["v"], s["k_exp"], s["v_exp"])
        h["batch"] = lib.KVBatch(s["cu"], s["kv"], s["table"], s["most"])
        h["out"] = torch.empty_like(s["q"])
        if c["op"] == "attention":
            h["lse"] = torch.empty(s["T"], c["hq"], dtype=torch.float32, device="cuda")
            h["ws"] = lib.new_kv_attention_workspace()
    return h


def run(s):
    c = s["case"]
    if own and "handles" not in s:
        s["handles"] = _handles(s)
    h = s.get("handles") if own else None
    if c["op"] == "rotary":
        if not own:
            return _rotate(s["x"], s["pos"], c["rot"], c["inter"], c["scaling"], c["factor"], c["inverse"])
        h["lib"].qspec_rotary(s["x"], s["pos"], h["rope"], h["out"], inverse=c["inverse"])
        return h["out"]
    if c["op"] == "append":
        if own:
            h["lib"].qspec_kv_append(h["cache"], h["batch"], s["k_new"], s["v_new"], rotary=h["rope"], q=s["q"], q_out=h["out"])
        q = h["out"] if own else _append(s)
        return {"q": q, "k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn),
                "k_exp": s["k_exp"], "v_exp": s["v_exp"]}
    if c["op"] == "attention":
        if not own:
            out, lse = _attention(s)
            return {"out": out, "lse": lse}
        h["lib"].qspec_kv_attention(h["cache"], h["batch"], s["q"], h["out"], h["ws"], window=c["window"], tree=s["tree"], lse=h["lse"])
        return {"out": h["out"], "lse": h["lse"]}
    if not own:
        return _logits(s)
    h["lib"].qspec_logits_adjust(s["logits"], h["out"], draft_tok=s["draft"], hist=s["hist"], hist_len=s["hist_len"],
                                 prompt_len=s["prompt_len"], penalties=s["pen"], bias_ids=s["bias_id"], bias=s["bias"], mask=s["mask"])
    return h["out"]


# ---------------------------------------------------------------------------------------- the definition, in 64 bits

def _turned(x, pos, rot, inter, scaling, factor, inverse):
    """Each pair as a complex number times exp(i angle), fp64."""
    n = rot // 2
    base = ROPE["base"] * (factor ** (rot / (rot - 2)) if scaling == "base" else 1.0)
    w = np.array([base ** (-2.0 * i / rot) for i in range(n)])
    mult = 1.0
    if scaling == "linear":
        w = w / factor
    elif scaling == "bands":
        for i in range(n):
            length = 2 * math.pi / w[i]
            if length > ROPE["orig"] / ROPE["low"]:
                w[i] /= factor
            elif length >= ROPE["orig"] / ROPE["high"]:
                f = (ROPE["orig"] / length - ROPE["low"]) / (ROPE["high"] - ROPE["low"])
                w[i] = (1 - f) * w[i] / factor + f * w[i]
    elif scaling == "yarn":
        at = [rot * math.log(ROPE["orig"] / (2 * math.pi * beta)) / (2 * math.log(base)) for beta in (ROPE["fast"], ROPE["slow"])]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        for i in range(n):
            r = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            w[i] = w[i] * ((1 - r) + r / factor)
        mult = 1 + 0.1 * math.log(factor) if factor > 1 else 1.0
    ang = torch.outer(pos.double(), torch.from_numpy(w).cuda())
    turn = torch.polar(torch.full_like(ang, mult), -ang if inverse else ang)[:, None]
    y = x.double().clone()
    head = y[..., :rot]
    pair = head.reshape(*head.shape[:-1], n, 2) if inter else torch.stack([head[..., :n], head[..., n:]], -1)
    z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
    y[..., :rot] = z.reshape(head.shape) if inter else torch.cat([z[..., 0], z[..., 1]], -1)
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _turned(s["x"], s["pos"], case["rot"], case["inter"], case["scaling"], case["factor"], case["inverse"])
    if case["op"] == "append":
        cu, kv = s["cu"].tolist(), s["kv"].tolist()
        pos = torch.cat([torch.arange(kv[b] - (cu[b + 1] - cu[b]), kv[b]) for b in range(case["B"])]).cuda()
        # codes are what the rounding gives, not computed numbers
        return {"q": _turned(s["q"], pos, case["dim"], case["inter"], case["scaling"], case["factor"], False),
                "k": None, "v": None, "k_exp": None, "v_exp": None}
    if case["op"] == "logits":
        x = s["logits"].double()
        B, G1, V = x.shape
        for b in range(B):
            hl, pl = int(s["hist_len"][b]), int(s["prompt_len"][b])
            rep, freq, pres = (float(t) for t in s["pen"][b])
            for i in range(G1):
                d = s["draft"][b, :i].long()
                c = torch.bincount(torch.cat([s["hist"][b, pl:hl].long(), d]), minlength=V)
                seen = torch.bincount(torch.cat([s["hist"][b, :hl].long(), d]), minlength=V) > 0
                r = x[b, i]
                r[seen] = torch.where(r[seen] > 0, r[seen] / rep, r[seen] * rep)
                r -= c * freq + (c > 0) * pres
                if s["bias_id"] is not None:
                    ok = s["bias_id"][b] >= 0
                    r[s["bias_id"][b][ok].long()] += s["bias"][b][ok].double()
                if s["mask"] is not None:
                    v = torch.arange(V, device="cuda")
                    r[(s["mask"][b, i].long()[v // 32] >> (v % 32)) % 2 == 0] = -math.inf
        return x
    B, Hk, G, D, P = case["B"], case["hk"], case["hq"] // case["hk"], case["dim"], case["page"]
    out = torch.zeros(s["T"], Hk * G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((s["T"], Hk * G), -math.inf, dtype=torch.float64, device="cuda")
    cu, kv = s["cu"].tolist(), s["kv"].tolist()
    for b in range(B):
        ids = s["table"][b, :-(-kv[b] // P)].long()
        n = cu[b + 1] - cu[b]
        for h in range(Hk):
            K, V = ((s[a][ids, h].view(torch.float8_e4m3fn).double() * 2.0 ** s[a + "_exp"][ids, h].double()[:, None, None])
                    .reshape(-1, D)[:kv[b]] for a in ("k", "v"))
            for t0 in range(0, n, 512):
                t1 = min(n, t0 + 512)
                i = torch.arange(t0, t1, device="cuda")[:, None] + kv[b] - n
                j = torch.arange(kv[b], device="cuda")[None]
                if s["tree"] is not None:
                    bits = s["tree"][cu[b] + t0:cu[b] + t1, None]
                    off = torch.where((j < kv[b] - n) | ((bits >> (j - (kv[b] - n)).clamp(min=0)) % 2 == 1), 0.0, -math.inf)
                else:
                    ok = (j <= i) & ((j > i - case["window"]) if case["window"] else (j >= 0))
                    off = torch.where(ok, 0.0, -math.inf)
                Q = s["q"][cu[b] + t0:cu[b] + t1, h * G:(h + 1) * G].double()
                S = torch.einsum("tgd,jd->tgj", Q, K) / D ** 0.5 + off[:, None].double()
                lse[cu[b] + t0:cu[b] + t1, h * G:(h + 1) * G] = torch.logsumexp(S, -1)
                out[cu[b] + t0:cu[b] + t1, h * G:(h + 1) * G] = torch.softmax(S, -1) @ V
    return {"out": out, "lse": lse}
