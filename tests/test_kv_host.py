"""Host side of the rotary, cache, attention and logits calls (no GPU): the frequency table against its
formulas, the refusals of the C ABI and of the binding, and the references' own rounding."""
import ctypes
import math
import random
from fractions import Fraction

import numpy as np
import pytest
import torch

import kv_ref as ref
from quantized_speculative_decoding_qspec_gb300 import qspec as q

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    return q.load()


@pytest.mark.parametrize("rot", [2, 6, 64, 96, 128])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("base", 8.0), ("bands", 8.0), ("yarn", 16.0), ("yarn", 1.0)])
def test_turns_follow_the_formulas(lib, rot, scaling, factor):
    if scaling == "base" and rot == 2:
        with pytest.raises(q.QSpecError, match="UNSUPPORTED_SHAPE"):
            q.qspec_rotary_turns(rot, 10000.0, scaling, factor)
        return
    args = dict(original=8192, low=1.0, high=4.0)
    if scaling == "yarn":
        args = dict(original=8192, low=1.0, high=32.0)
    turns, mult = q.qspec_rotary_turns(rot, 500000.0, scaling, factor, **args)
    w, m = ref.frequencies(rot, 500000.0, scaling, factor, original=8192)
    assert abs(mult - m) <= 2 ** -24 * m
    got = turns.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64 * 2 * math.pi
    # each word: a few fp64 roundings of pow, log and the scaling (16 of them), and 2^-64 turns
    assert np.all(np.abs(got - np.array(w)) <= 16 * 2.0 ** -53 * np.array(w) + 2 * math.pi * 2.0 ** -64)


def test_angle_of_a_far_position_is_the_fraction_of_a_turn(lib):
    turns, _ = q.qspec_rotary_turns(128, 10000.0)
    word = int(turns.numpy().view(np.uint64)[3])
    for pos in (1, 8191, 2 ** 31 - 1, -5):
        exact = Fraction(pos * word, 2 ** 64) % 1
        assert Fraction((pos * word) % 2 ** 64, 2 ** 64) == exact


def test_turns_refusals(lib):
    f = lib.qspec_rotary_turns
    buf = (ctypes.c_uint64 * 64)()
    m = ctypes.c_float()
    p, mp = ctypes.addressof(buf), ctypes.addressof(m)
    assert f(128, 10000.0, 0, 1.0, 0.0, 0.0, 0.0, p, mp) == 0
    assert f(128, 10000.0, 0, 1.0, 0.0, 0.0, 0.0, None, mp) == 1
    assert f(128, 1.0, 0, 1.0, 0.0, 0.0, 0.0, p, mp) == 1            # base not above 1
    assert f(128, float("nan"), 0, 1.0, 0.0, 0.0, 0.0, p, mp) == 1
    assert f(128, 10000.0, 5, 1.0, 0.0, 0.0, 0.0, p, mp) == 1        # no such scaling
    assert f(128, 10000.0, 1, 0.5, 0.0, 0.0, 0.0, p, mp) == 1        # factor below 1
    assert f(128, 10000.0, 3, 2.0, 0.0, 1.0, 4.0, p, mp) == 1        # no trained length
    assert f(128, 10000.0, 3, 2.0, 8192.0, 4.0, 4.0, p, mp) == 1     # empty band
    assert f(7, 10000.0, 0, 1.0, 0.0, 0.0, 0.0, p, mp) == 2
    assert f(1026, 10000.0, 0, 1.0, 0.0, 0.0, 0.0, p, mp) == 2
    with pytest.raises(ValueError, match="scaling"):
        q.qspec_rotary_turns(128, scaling="other")


def plan(**kw):
    d = dict(turns=FAKE, rot=64, interleaved=0, mult=1.0, reserved=0)
    d.update(kw)
    return ctypes.byref(q.RotaryPlan(*(d[k] for k in ("turns", "rot", "interleaved", "mult", "reserved"))))


def test_rotary_refusals(lib):
    f = lib.qspec_rotary
    ok = dict(x=FAKE, xt=1024, xh=128, pos=FAKE, T=4, H=8, D=128, plan=plan(), inv=0, out=FAKE, ot=1024, oh=128)

    def call(**kw):
        d = {**ok, **kw}
        return f(d["x"], d["xt"], d["xh"], d["pos"], d["T"], d["H"], d["D"], d["plan"], d["inv"], d["out"], d["ot"], d["oh"], None)

    for name in ("x", "pos", "plan", "out"):
        assert call(**{name: None}) == 1, name
    assert call(T=0) == 1 and call(H=0) == 1 and call(D=0) == 1
    assert call(plan=plan(turns=None)) == 1 and call(plan=plan(reserved=3)) == 1
    assert call(plan=plan(mult=float("inf"))) == 1
    assert call(D=100) == 2 and call(D=1032) == 2 and call(H=65536) == 2
    assert call(plan=plan(rot=130)) == 2 and call(plan=plan(rot=63)) == 2 and call(plan=plan(rot=0)) == 2
    assert call(xt=-8) == 2 and call(xt=1 << 39) == 2
    assert call(x=FAKE + 8) == 3 and call(out=FAKE + 2) == 3 and call(pos=FAKE + 2) == 3
    assert call(xt=1028) == 3 and call(oh=132) == 3 and call(plan=plan(turns=FAKE + 4)) == 3


def cache(**kw):
    d = dict(k=FAKE, v=FAKE, k_exp=FAKE, v_exp=FAKE, n_pages=10, heads=8, page=64, dim=128, reserved=0)
    d.update(kw)
    return ctypes.byref(q.KVCacheDesc(*d.values()))


def batch(**kw):
    d = dict(cu_tok=FAKE, kv_len=FAKE, pages=FAKE, B=2, max_pages=4, max_tok=3, reserved=0, T=6)
    d.update(kw)
    return ctypes.byref(q.KVBatchDesc(*d.values()))


BAD_KV = [(dict(c=None), 1), (dict(b=None), 1), (dict(c=dict(k=None)), 1), (dict(c=dict(v_exp=None)), 1),
          (dict(b=dict(cu_tok=None)), 1), (dict(b=dict(pages=None)), 1), (dict(c=dict(reserved=1)), 1),
          (dict(b=dict(reserved=1)), 1), (dict(c=dict(n_pages=0)), 1), (dict(c=dict(heads=0)), 1), (dict(b=dict(B=0)), 1),
          (dict(b=dict(T=0)), 1), (dict(b=dict(max_tok=0)), 1), (dict(b=dict(max_pages=0)), 1),
          (dict(c=dict(page=48)), 2), (dict(c=dict(dim=96)), 2), (dict(b=dict(B=1025)), 2), (dict(b=dict(max_tok=7)), 2),
          (dict(b=dict(max_pages=1 << 25)), 2), (dict(b=dict(max_pages=(1 << 24) + 1)), 2), (dict(c=dict(heads=4097)), 2),
          (dict(c=dict(k=FAKE + 8)), 3), (dict(b=dict(kv_len=FAKE + 2)), 3)]


def kv_args(kw):
    c, b = kw.get("c", {}), kw.get("b", {})
    return cache(**c) if c is not None else None, batch(**b) if b is not None else None


@pytest.mark.parametrize("kw,code", BAD_KV)
def test_cache_and_batch_refusals(lib, kw, code):
    c, b = kv_args(kw)
    assert lib.qspec_kv_append(c, b, FAKE, 1024, FAKE, 1024, None, None, None, 0, 0, None, 0, None) == code
    assert lib.qspec_kv_attention(c, b, FAKE, 4096, 32, 0.1, 0, None, FAKE, 4096, None, FAKE, 1 << 40, None) == code


def test_append_refusals(lib):
    ok = dict(k=FAKE, ks=1024, v=FAKE, vs=1024, plan=plan(), pos=None, q=FAKE, qs=4096, hq=32, qo=FAKE, qos=4096)

    def call(**kw):
        d = {**ok, **kw}
        return lib.qspec_kv_append(cache(), batch(), d["k"], d["ks"], d["v"], d["vs"], d["plan"], d["pos"], d["q"], d["qs"],
                                   d["hq"], d["qo"], d["qos"], None)

    assert call(k=None) == 1 and call(v=None) == 1 and call(qo=None) == 1 and call(hq=0) == 1
    assert call(plan=plan(turns=None)) == 1
    assert call(ks=1016) == 2 and call(vs=0) == 2 and call(hq=33) == 2 and call(qs=4088) == 2 and call(qos=8) == 2
    assert call(plan=plan(rot=40)) == 2                                # half layout: a multiple of 16
    assert call(plan=plan(rot=130)) == 2
    assert call(k=FAKE + 2) == 3 and call(ks=1028) == 3 and call(q=FAKE + 8) == 3 and call(pos=FAKE + 1) == 3


def test_attention_refusals(lib):
    W = lib.qspec_kv_attention_workspace_size()
    assert W > 0
    ok = dict(q=FAKE, qs=4096, hq=32, scale=0.1, window=0, tree=None, out=FAKE, os=4096, lse=None, ws=FAKE, W=W, b={})

    def call(**kw):
        d = {**ok, **kw}
        return lib.qspec_kv_attention(cache(), batch(**d["b"]), d["q"], d["qs"], d["hq"], d["scale"], d["window"], d["tree"],
                                      d["out"], d["os"], d["lse"], d["ws"], d["W"], None)

    assert call(q=None) == 1 and call(out=None) == 1 and call(hq=0) == 1 and call(window=-1) == 1
    assert call(scale=float("nan")) == 1 and call(scale=float("inf")) == 1
    assert call(hq=12) == 2 and call(hq=8 * 129, qs=8 * 129 * 128, os=8 * 129 * 128) == 2 and call(qs=4088) == 2
    assert call(tree=FAKE, window=4) == 2
    assert call(tree=FAKE, b=dict(max_tok=65, T=80)) == 2
    assert call(q=FAKE + 2) == 3 and call(os=4100) == 3 and call(tree=FAKE + 4) == 3 and call(lse=FAKE + 2) == 3
    assert call(ws=FAKE + 8) == 3
    assert call(ws=None) == 4 and call(W=W - 1) == 4


def test_logits_refusals(lib):
    ok = dict(x=FAKE, B=2, rows=4, V=1000, d=FAKE, h=FAKE, hs=10, hl=FAKE, pl=FAKE, pen=FAKE, bi=FAKE, bv=FAKE, nb=3, m=FAKE, out=FAKE)

    def call(**kw):
        d = {**ok, **kw}
        return lib.qspec_logits_adjust(*(d[k] for k in ok), None)

    assert call(x=None) == 1 and call(out=None) == 1 and call(B=0) == 1 and call(rows=0) == 1 and call(V=0) == 1
    assert call(h=None) == 1 and call(hl=None) == 1 and call(hs=0) == 1          # history without its lengths
    assert call(h=None, hl=None) == 1                                            # prompt lengths without a history
    assert call(bi=None) == 1 and call(bv=None) == 1 and call(nb=0) == 1
    assert call(rows=18) == 2 and call(V=1) == 2 and call(V=(1 << 24) + 1) == 2 and call(B=65536) == 2
    assert call(x=FAKE + 2) == 3 and call(out=FAKE + 8) == 3
    for name in ("d", "h", "hl", "pl", "pen", "bi", "bv", "m"):
        assert call(**{name: FAKE + 2}) == 3, name


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses_wrong_types_and_short_buffers():
    x, pos = z(4, 2, 64), z(4, dtype=torch.int32)
    with pytest.raises(TypeError, match="pos must be"):
        q.qspec_rotary(x, pos.long(), None, x)
    with pytest.raises(ValueError, match="x and out"):
        q.qspec_rotary(x, pos, None, z(4, 2, 32))
    with pytest.raises(ValueError, match="live on the GPU"):
        q.qspec_rotary(x, pos, None, x)
    with pytest.raises(TypeError, match="k must be"):
        q.KVCache(z(2, 2, 16, 64), z(2, 2, 16, 64), z(2, 2, dtype=torch.int8), z(2, 2, dtype=torch.int8))
    u = z(2, 2, 16, 64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="k_exp holds 3 elements"):
        q.KVCache(u, u, z(3, dtype=torch.int8), z(4, dtype=torch.int8))
    with pytest.raises(ValueError, match="must be \\[pages"):
        q.KVCache(u, u[:1], z(4, dtype=torch.int8), z(4, dtype=torch.int8))
    with pytest.raises(ValueError, match="cu_tok holds"):
        q.KVBatch(z(2, dtype=torch.int32), z(2, dtype=torch.int32), z(2, 3, dtype=torch.int32), 1)
    L = z(2, 3, 40)
    with pytest.raises(ValueError, match="out holds"):
        q.qspec_logits_adjust(L, z(2, 3, 39))
    with pytest.raises(ValueError, match="mask holds"):
        q.qspec_logits_adjust(L, L, mask=z(2, 3, 1, dtype=torch.int32))
    with pytest.raises(ValueError, match="draft_tok holds"):
        q.qspec_logits_adjust(L, L, draft_tok=z(2, 1, dtype=torch.int32))
    with pytest.raises(ValueError, match="penalties holds"):
        q.qspec_logits_adjust(L, L, penalties=z(5, dtype=torch.float32))
    with pytest.raises(ValueError, match="hist must be"):
        q.qspec_logits_adjust(L, L, hist=z(5, dtype=torch.int32), hist_len=z(2, dtype=torch.int32))


def test_reference_rounding_is_e4m3():
    """The references' e4m3 codes: every code reads back to itself, ties go to even, large values saturate."""
    codes = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F], dtype=torch.uint8)
    vals = ref.e4m3_value(codes)
    assert torch.equal(ref.e4m3(vals), codes)
    assert float(vals.max()) == 448.0
    assert torch.equal(vals.float(), codes.view(torch.float8_e4m3fn).float())
    x = torch.tensor([1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, 1e9, -460.0, 0.3], dtype=torch.float64)
    want = [1.0, 1.25, 0.0, 2.0 ** -8, 448.0, -448.0, 0.3125]
    assert ref.e4m3_value(ref.e4m3(x)).tolist() == want
    r = random.Random(5)
    for _ in range(200):
        a = r.uniform(0, 500) * 2.0 ** r.randint(-6, 6)
        e = ref.block_exp(a)
        assert a <= 448 * 2.0 ** e and (e == -40 or a > 448 * 2.0 ** (e - 1))
