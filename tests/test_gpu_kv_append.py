"""qspec_kv_append: codes and exponents bit-exact against the definition; rotated keys and queries within the
rotation's tolerance."""
import pytest
import torch

import kv_ref as ref
from gpu_util import DEV, lib

pytestmark = pytest.mark.gpu


def new_rows(g, T, H, D, pad=0, scale=None):
    buf = torch.randn(T, H * D + pad, generator=g)
    if scale is not None:
        buf = buf * torch.exp2(scale * torch.randn(T, 1, generator=g))
    return buf.to(torch.bfloat16)


CASES = [  # tok, kv after the append, heads, page, dim
    ([1], [1], 1, 16, 64), ([1], [517], 8, 64, 128), ([4, 4, 4], [4, 66, 130], 2, 64, 128), ([1, 3, 0, 5], [16, 17, 40, 33], 3, 16, 64),
    ([130, 1, 64], [130, 128, 64], 2, 32, 128), ([257, 2], [300, 2], 1, 128, 128), ([40, 31, 128], [41, 160, 129], 2, 128, 64)]


@pytest.mark.parametrize("tok,kv,H,P,D", CASES)
def test_codes_are_exact(tok, kv, H, P, D):
    q = lib()
    bt = ref.Batch(7 + P + D, tok, kv, H, P, D)
    g = torch.Generator().manual_seed(1)
    # keys vary a lot from token to token, so pages grow and are quantised again
    k, v = new_rows(g, bt.T, H, D, 0, 6.0), new_rows(g, bt.T, H, D, 8, 0.5)
    cache, batch = bt.gpu(q)
    kg, vg = k.to(DEV).view(bt.T, H, D), v.to(DEV)[:, :H * D].unflatten(1, (H, D))
    q.qspec_kv_append(cache, batch, kg, vg)
    q.qspec_check_status()
    for side, new in (("k", k.view(bt.T, H, D)), ("v", v[:, :H * D].reshape(bt.T, H, D))):
        codes, exps = bt.codes[side].clone(), bt.exps[side].clone()
        ref.append(codes, exps, new, bt.table, bt.cu, bt.kv)
        got_c, got_e = (cache.k, cache.k_exp) if side == "k" else (cache.v, cache.v_exp)
        assert torch.equal(got_e.cpu(), exps)
        # the slots behind a sequence's end are never read: only those up to it must agree
        valid = torch.zeros(bt.n_pages, P, dtype=torch.bool)
        for b in range(bt.B):
            for p in range(kv[b]):
                valid[int(bt.table[b, p // P]), p % P] = True
        sel = valid[:, None, :, None].expand_as(codes)
        assert torch.equal(got_c.cpu()[sel], codes[sel])
        assert torch.equal(got_c.cpu()[~sel], codes[~sel])      # nothing else is touched
    # once more: the same tokens at the same place change nothing
    before = [t.clone() for t in (cache.k, cache.v, cache.k_exp, cache.v_exp)]
    q.qspec_kv_append(cache, batch, kg, vg)
    assert all(torch.equal(a, b) for a, b in zip(before, (cache.k, cache.v, cache.k_exp, cache.v_exp)))


@pytest.mark.parametrize("D,P", [(64, 16), (128, 64), (128, 128)])
def test_edges_of_the_scale(D, P):
    """Zeros, the largest value that still takes an exponent and the next one, tiny and huge values."""
    q = lib()
    edge = [0.0, 448.0, 450.0, 1.75, 1.7578125, 2.0 ** -60, 3e38, 2.0 ** -40 * 448, -448.0 * 2 ** 40, 1e-30]
    bt = ref.Batch(3, [1] * len(edge), [1] * len(edge), 1, P, D)
    g = torch.Generator().manual_seed(2)
    x = torch.rand(len(edge), 1, D, generator=g) * 2 - 1
    x[:, 0, 5] = 1.0
    x = (x.double() * torch.tensor(edge, dtype=torch.float64)[:, None, None]).to(torch.bfloat16)
    cache, batch = bt.gpu(q)
    q.qspec_kv_append(cache, batch, x.to(DEV), (-x).to(DEV))
    q.qspec_check_status()
    for side, new in (("k", x), ("v", -x)):
        codes, exps = bt.codes[side].clone(), bt.exps[side].clone()
        ref.append(codes, exps, new, bt.table, bt.cu, bt.kv)
        assert torch.equal((cache.k if side == "k" else cache.v).cpu(), codes)
        assert torch.equal((cache.k_exp if side == "k" else cache.v_exp).cpu(), exps)


def test_rejected_tokens_are_written_over():
    """A verify step appends gamma + 1 tokens, keeps two, and the next step starts after those."""
    q = lib()
    H, P, D = 2, 16, 64
    bt = ref.Batch(11, [4], [18], H, P, D)
    g = torch.Generator().manual_seed(4)
    cache, batch = bt.gpu(q)
    codes = {s: bt.codes[s].clone() for s in "kv"}
    exps = {s: bt.exps[s].clone() for s in "kv"}
    for kv in (18, 20, 21, 25):      # 14 + 4, 16 + 4, 17 + 4, 21 + 4 positions
        k, v = (new_rows(g, 4, H, D, 0, 4.0).view(4, H, D) for _ in range(2))
        batch.kv_len.fill_(kv)
        q.qspec_kv_append(cache, batch, k.to(DEV), v.to(DEV))
        for s, new in (("k", k), ("v", v)):
            ref.append(codes[s], exps[s], new, bt.table, [0, 4], [kv])
    q.qspec_check_status()
    used = bt.table[0].long()
    for s, c, e in (("k", cache.k, cache.k_exp), ("v", cache.v, cache.v_exp)):
        assert torch.equal(e.cpu()[used], exps[s][used])
        flat = c.cpu()[used].permute(1, 0, 2, 3).reshape(H, -1, D)[:, :25]
        assert torch.equal(flat, codes[s][used].permute(1, 0, 2, 3).reshape(H, -1, D)[:, :25])


@pytest.mark.parametrize("D,rot,inter,hq,own_pos", [(64, 64, False, 4, False), (128, 96, False, 12, True), (128, 50, True, 2, False),
                                                    (64, 16, True, 14, True), (128, 128, False, 64, False)])
def test_rotation_on_the_way(D, rot, inter, hq, own_pos):
    q = lib()
    H, P, tok, kv = 2, 32, [5, 40, 1], [37, 40, 65]
    bt = ref.Batch(21, tok, kv, H, P, D)
    g = torch.Generator().manual_seed(6)
    T = bt.T
    k, v, qq = new_rows(g, T, H, D).view(T, H, D), new_rows(g, T, H, D).view(T, H, D), new_rows(g, T, hq, D).view(T, hq, D)
    pos = torch.tensor([kv[b] - tok[b] + i for b in range(3) for i in range(tok[b])], dtype=torch.int32)
    if own_pos:
        pos = pos * 3 + 1000
    rope = q.Rotary(rot, interleaved=inter)
    w, mult = ref.frequencies(rot, 10000.0)
    cache, batch = bt.gpu(q)
    qg = qq.to(DEV)
    q_out = torch.empty_like(qg)
    q.qspec_kv_append(cache, batch, k.to(DEV), v.to(DEV), rotary=rope, pos=pos.to(DEV) if own_pos else None, q=qg, q_out=q_out)
    q.qspec_check_status()
    want, size = ref.rotate(qq, pos, w, mult, inter)
    assert bool(((q_out.double().cpu() - want).abs() <= ref.BF16 * want.abs() + 2.0 ** -21 * size).all())
    in_place = qg.clone()
    q.qspec_kv_append(cache, batch, k.to(DEV), v.to(DEV), rotary=rope, pos=pos.to(DEV) if own_pos else None, q=in_place)
    assert torch.equal(in_place, q_out)
    # keys: rotated and rounded to bf16, then e4m3 under the page's scale; the page's exponent from the rotated keys
    kw, ks = ref.rotate(k, pos, w, mult, inter)
    t = 0
    for b in range(3):
        for i in range(tok[b]):
            p = kv[b] - tok[b] + i
            page = int(bt.table[b, p // P])
            e = cache.k_exp[page].cpu().double()
            got = ref.e4m3_value(cache.k[page, :, p % P].cpu()) * torch.exp2(e)[:, None]
            tol = (ref.E4M3 + 2 * ref.BF16) * kw[t].abs() + 2.0 ** -20 * ks[t] + 2.0 ** -10 * torch.exp2(e)[:, None]
            assert bool(((got - kw[t]).abs() <= tol).all())
            assert bool((kw[t].abs().amax(1) <= 448 * torch.exp2(e) * (1 + 2 * ref.BF16)).all())
            t += 1


def test_same_keys_as_the_rotary_call():
    """Keys rotated on the way and keys rotated by qspec_rotary first differ by bf16 roundings at most."""
    q = lib()
    H, P, D = 4, 64, 128
    bt = ref.Batch(5, [64], [64], H, P, D)
    g = torch.Generator().manual_seed(8)
    k = new_rows(g, 64, H, D).view(64, H, D).to(DEV)
    rope = q.Rotary(128, 500000.0)
    pos = torch.arange(64, dtype=torch.int32, device=DEV)
    one, batch = bt.gpu(q)
    two, _ = bt.gpu(q)
    q.qspec_kv_append(one, batch, k, k, rotary=rope)
    r = torch.empty_like(k)
    q.qspec_rotary(k, pos, rope, r)
    q.qspec_kv_append(two, batch, r, k)
    q.qspec_check_status()
    page = int(bt.table[0, 0])
    a, b = one.values("k")[page], two.values("k")[page]
    assert torch.equal(one.v[page], two.v[page])
    assert float((a - b).abs().max()) <= 2 * ref.E4M3 * float(b.abs().max())
    assert float((a != b).float().mean()) < 1e-3


def test_bad_values_are_reported_and_harmless():
    q = lib()
    H, P, D = 2, 16, 64
    bt = ref.Batch(13, [2, 2, 2, 2], [20, 18, 33, 17], H, P, D)
    g = torch.Generator().manual_seed(5)
    k = new_rows(g, 8, H, D).view(8, H, D)
    v = k.clone()
    k[1, 0, 3], v[1, 1, 7], v[0, 0, 0] = float("nan"), float("inf"), float("-inf")
    cache, batch = bt.gpu(q)
    batch.pages[1, 1] = bt.n_pages           # an id just behind the cache
    batch.pages[2, 2] = -1                   # the third sequence's last page (its only new token there)
    batch.kv_len[3] = 1                      # fewer positions than new tokens
    q.qspec_kv_append(cache, batch, k.to(DEV), v.to(DEV))
    with pytest.raises(q.QSpecError, match="INVALID_ARG"):
        q.qspec_check_status()
    q.qspec_check_status()                   # reported once
    k0, v0 = torch.where(k.isfinite(), k, 0), torch.where(v.isfinite(), v, 0)
    for side, new, c, e in (("k", k0, cache.k, cache.k_exp), ("v", v0, cache.v, cache.v_exp)):
        codes, exps = bt.codes[side].clone(), bt.exps[side].clone()
        ref.append(codes, exps, new[:2], bt.table[:1], [0, 2], [20])
        # the third sequence: position 31 (page 1) is written, 32 is not
        ref.append(codes, exps, new[4:5], bt.table[2:3], [0, 1], [32])
        assert torch.equal(c.cpu(), codes) and torch.equal(e.cpu(), exps)


def test_ranges_of_the_batch_are_checked():
    q = lib()
    bt = ref.Batch(17, [3, 3], [10, 12], 1, 16, 64)
    k = torch.ones(6, 1, 64, dtype=torch.bfloat16, device=DEV)
    for name, at, val in (("cu_tok", 1, 7), ("cu_tok", 1, -1), ("kv_len", 0, -3), ("kv_len", 1, 1 << 20), ("cu_tok", 2, 9)):
        cache, batch = bt.gpu(q)
        getattr(batch, name)[at] = val
        q.qspec_kv_append(cache, batch, k, k)
        with pytest.raises(q.QSpecError, match="INVALID_ARG"):
            q.qspec_check_status()
    cache, batch = bt.gpu(q)
    batch.desc.max_tok = 2                   # a promise that a sequence breaks
    q.qspec_kv_append(cache, batch, k, k)
    with pytest.raises(q.QSpecError, match="INVALID_ARG"):
        q.qspec_check_status()
    assert torch.equal(cache.k.cpu(), bt.codes["k"])
