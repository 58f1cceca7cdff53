"""Plain 64-bit references (torch, CPU) of the rotary, cache, attention and logits calls, and the
inputs of their tests.  Written from the definitions in include/qspec.h; nothing of the library is used."""
import math

import numpy as np
import torch

BF16, E4M3 = 2.0 ** -8, 2.0 ** -4   # half a step, relative (e4m3: of a normal code)


def frequencies(rot, base, scaling="none", factor=1.0, original=0.0, low=1.0, high=4.0, slow=1.0, fast=32.0):
    """([rot/2] radians per position, fp64 list; factor on the rotated values)."""
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    w = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [x / factor for x in w], 1.0
    if scaling == "bands":
        def band(x):
            turns = original * x / (2 * math.pi)
            if turns <= low:
                return x / factor
            if turns >= high:
                return x
            keep = (turns - low) / (high - low)
            return (1 - keep) * x / factor + keep * x
        return [band(x) for x in w], 1.0
    if scaling == "yarn":
        def index(turns):
            return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        first, last = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), rot - 1)
        ramp = [min(max((i - first) / max(last - first, 1e-3), 0.0), 1.0) for i in range(rot // 2)]
        return [x / factor * r + x * (1 - r) for x, r in zip(w, ramp)], 0.1 * math.log(factor) + 1
    return w, 1.0


def rotate(x, pos, w, mult, interleaved, inverse=False):
    """x [T, H, D], pos [T] -> (rotated fp64, |a| + |b| of each value's pair: what rounding errors scale with)."""
    x = x.double().cpu()
    ang = torch.outer(pos.double().cpu(), torch.tensor(w, dtype=torch.float64)) * (-1 if inverse else 1)
    c, s = (ang.cos() * mult)[:, None], (ang.sin() * mult)[:, None]
    n = len(w)
    y, size = x.clone(), x.abs()
    ia = torch.arange(n) * 2 if interleaved else torch.arange(n)
    ib = ia + 1 if interleaved else ia + n
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    size[..., ia] = size[..., ib] = (a.abs() + b.abs()) * mult
    return y, size


def block_exp(amax):
    """The smallest e with amax <= 448 * 2^e, within -40 .. 40."""
    if amax == 0:
        return -40
    e = -41
    while amax > 448.0 * 2.0 ** e and e < 40:
        e += 1
    return max(e, -40)


def e4m3(x):
    """fp64 tensor -> e4m3 codes: nearest, ties to even, saturating.  By the list of the 127 finite magnitudes."""
    mags = torch.tensor([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:119],
                        dtype=torch.float64)
    a = x.abs().clamp(max=448.0)
    hi = torch.searchsorted(mags, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    d_hi, d_lo = mags[hi] - a, a - mags[lo]
    take_lo = (d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0))
    code = torch.where(take_lo, lo, hi)
    sign = torch.signbit(x).to(torch.int64) * 128
    return (code + sign).to(torch.uint8)


def e4m3_value(code):
    c = code.to(torch.int64)
    e, m = (c >> 3) & 15, c & 7
    v = torch.where(e == 0, m.double() * 2.0 ** -9, (8 + m).double() * torch.pow(2.0, (e - 10).double()))
    return torch.where(c >= 128, -v, v)


def append(codes, exps, new, table, cu, kv):
    """Writes new [T, H, D] (values already rotated and rounded to bf16) into codes [n, H, P, D] / exps [n, H]."""
    n, H, P, D = codes.shape
    for b in range(len(kv)):
        cnt = cu[b + 1] - cu[b]
        start = kv[b] - cnt
        for pg in sorted({(start + i) // P for i in range(cnt)}):
            lo, hi = max(start, pg * P), min(kv[b], (pg + 1) * P)
            page = int(table[b, pg])
            for h in range(H):
                x = new[cu[b] + lo - start:cu[b] + hi - start, h].double()
                e = block_exp(float(x.abs().max()))
                if lo > pg * P:
                    old = int(exps[page, h])
                    e = max(e, old)
                    if e > old:
                        seg = codes[page, h, :lo - pg * P]
                        codes[page, h, :lo - pg * P] = e4m3(e4m3_value(seg) * 2.0 ** (old - e))
                exps[page, h] = e
                codes[page, h, lo - pg * P:hi - pg * P] = e4m3(x * 2.0 ** -e)


class Batch:
    """Random sequences in a shuffled paged cache whose unused slots hold the worst stale bytes."""

    def __init__(self, seed, tok, kv, heads, page, dim, spread=2.0, spare=3):
        g = torch.Generator().manual_seed(seed)
        self.tok, self.kv, self.H, self.P, self.D = list(tok), list(kv), heads, page, dim
        self.B, self.T = len(tok), sum(tok)
        self.cu = [0] + [int(x) for x in np.cumsum(tok)]
        need = [-(-n // page) for n in kv]
        self.n_pages = sum(need) + spare
        perm = torch.randperm(self.n_pages, generator=g).to(torch.int32)
        self.table = torch.full((self.B, max(max(need), 1)), -7, dtype=torch.int32)  # never read beyond kv
        self.codes = {}
        self.exps = {}
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        for side in "kv":
            codes = torch.full((self.n_pages, heads, page, dim), 0x7F, dtype=torch.uint8)   # NaN codes
            exps = torch.full((self.n_pages, heads), 99, dtype=torch.int8)
            x = torch.randn(self.n_pages, heads, page, dim, generator=g, dtype=torch.float64)
            x = x * torch.exp2(spread * torch.randn(self.n_pages, heads, 1, 1, generator=g, dtype=torch.float64))
            for b, n in enumerate(self.kv):
                for pg in range(need[b]):
                    p, used = int(self.table[b, pg]), min(page, n - pg * page)
                    for h in range(heads):
                        v = x[p, h, :used].to(torch.bfloat16).double()
                        e = block_exp(float(v.abs().max()))
                        exps[p, h] = e
                        codes[p, h, :used] = e4m3(v * 2.0 ** -e)
            self.codes[side], self.exps[side] = codes, exps

    def values(self, side, b):
        """[H, kv, D] fp64 values of sequence b."""
        ids = self.table[b, :-(-self.kv[b] // self.P)].long()
        x = e4m3_value(self.codes[side][ids]) * torch.exp2(self.exps[side][ids].double())[..., None, None]
        return x.permute(1, 0, 2, 3).reshape(self.H, -1, self.D)[:, :self.kv[b]]

    def gpu(self, q):
        """(KVCache, KVBatch) on the GPU."""
        d = "cuda"
        cache = q.KVCache(self.codes["k"].to(d), self.codes["v"].to(d), self.exps["k"].to(d), self.exps["v"].to(d))
        batch = q.KVBatch(torch.tensor(self.cu, dtype=torch.int32, device=d), torch.tensor(self.kv, dtype=torch.int32, device=d),
                          self.table.to(d), max(max(self.tok), 1))
        return cache, batch


def visible(i, n, kv, window=0, bits=None):
    """Truth values over the kv positions that new token i of n sees."""
    j = torch.arange(kv)
    base = kv - n
    if bits is not None:
        return torch.tensor([x < base or bool((bits >> (x - base)) & 1) for x in range(kv)], dtype=torch.bool)
    see = j <= base + i
    return see & (j > base + i - window) if window else see


def attention(bt, q, scale, window=0, tree=None):
    """fp64 (out [T, Hq, D], lse [T, Hq], tolerance of out, tolerance of lse).

    The tolerances count, per output: its own rounding to bf16 (half a step); the rounding of the
    probabilities to fp16 (2^-11 each, 2^-25 of the largest weight p * 2^exp below fp16's normal range,
    taken on the codes); the scores' fp32 error, at most D + 2 roundings of the summed magnitudes,
    which enters the probabilities twice (numerator and denominator); and fp32 sums over the keys.
    """
    T, Hq, D = q.shape
    G = Hq // bt.H
    out, tol = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
    lse, tol_l = torch.full((T, Hq), -math.inf, dtype=torch.float64), torch.zeros(T, Hq, dtype=torch.float64)
    qd = q.double().cpu()
    for b in range(bt.B):
        n, kv = bt.tok[b], bt.kv[b]
        if n == 0 or kv == 0:
            continue
        K, V = bt.values("k", b), bt.values("v", b)
        ids = bt.table[b, :-(-kv // bt.P)].long()
        unit = torch.exp2(bt.exps["v"][ids].double()).repeat_interleave(bt.P, 0)[:kv]   # [kv, H] scale of each value
        for i in range(n):
            t = bt.cu[b] + i
            see = visible(i, n, kv, window, None if tree is None else int(tree[t]) & (2 ** 64 - 1))
            if not bool(see.any()):
                continue
            for h in range(Hq):
                k, v, u = K[h // G][see], V[h // G][see], unit[see, h // G]
                s = scale * (k @ qd[t, h])
                m = s.max()
                p = torch.exp(s - m)
                l = p.sum()
                out[t, h] = (p @ v) / l
                lse[t, h] = m + torch.log(l)
                es = abs(scale) * float((k.abs() @ qd[t, h].abs()).max()) * (D + 2) * 2.0 ** -24
                many = (len(s) + 64) * 2.0 ** -24
                mag = (p @ v.abs()) / l
                w = (p * u).max()
                tiny = 2.0 ** -25 * w * (v.abs() / u[:, None]).sum(0) / l
                tol[t, h] = BF16 * out[t, h].abs() + (2.0 ** -11 + 2 * es + many + 2.0 ** -20) * mag * 1.01 + tiny
                tol_l[t, h] = es + many + 2.0 ** -20 + 2.0 ** -22 * abs(float(lse[t, h]))
    return out, lse, tol, tol_l


def logits(x, draft=None, hist=None, hist_len=None, prompt_len=None, pen=None, bias_ids=None, bias=None, mask=None):
    """fp64 adjusted logits [B, rows, V], and whether each one was touched."""
    B, R, V = x.shape
    z, touched = x.double().clone(), torch.zeros(B, R, V, dtype=torch.bool)
    for b in range(B):
        for i in range(R):
            made, seen = torch.zeros(V, dtype=torch.int64), torch.zeros(V, dtype=torch.bool)
            if hist is not None:
                for k in range(int(hist_len[b])):
                    v = int(hist[b, k])
                    if 0 <= v < V:
                        seen[v] = True
                        if k >= (int(prompt_len[b]) if prompt_len is not None else 0):
                            made[v] += 1
            if draft is not None:
                for v in draft[b, :i].tolist():
                    if 0 <= v < V:
                        seen[v] = True
                        made[v] += 1
            r = z[b, i]
            if pen is not None:
                rep, freq, pres = (float(t) for t in pen[b])
                if not rep > 0:
                    rep = 1.0
                r[seen] = torch.where(r[seen] > 0, r[seen] / rep, r[seen] * rep)
                r -= freq * made + pres * (made > 0)
                touched[b, i] |= seen
            if bias is not None:
                last = {}
                for v, w in zip(bias_ids[b].tolist(), bias[b].tolist()):
                    if 0 <= v < V:
                        last[v] = w
                for v, w in last.items():
                    r[v] += w
                    touched[b, i, v] = True
            if mask is not None:
                for v in range(V):
                    if not (int(mask[b, i, v // 32]) >> (v % 32)) & 1:
                        r[v] = -math.inf
                        touched[b, i, v] = True
    return z, touched
