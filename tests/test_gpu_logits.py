"""qspec_logits_adjust against the definition in 64 bits.

Tolerance: half a bf16 step of the result, and five fp32 roundings (division or product, penalty product and
sum, the difference, the bias) of values no larger than |logit| * rep + freq * count + presence + |bias| <= 64 here."""
import pytest
import torch

import kv_ref as ref
from gpu_util import DEV, lib

pytestmark = pytest.mark.gpu


def inputs(seed, B, R, V, hist, n_bias, with_mask):
    g = torch.Generator().manual_seed(seed)
    x = (4 * torch.randn(B, R, V, generator=g)).to(torch.bfloat16)
    d = {"draft": torch.randint(0, V, (B, max(R - 1, 0)), generator=g, dtype=torch.int32)}
    if hist:
        d["hist"] = torch.randint(0, min(V, 97), (B, hist), generator=g, dtype=torch.int32)
        d["hist_len"] = torch.randint(0, hist + 1, (B,), generator=g, dtype=torch.int32)
        d["hist_len"][0] = hist
        d["prompt_len"] = (d["hist_len"].float() * torch.rand(B, generator=g)).to(torch.int32)
        d["draft"][:, :] = torch.where(torch.rand(d["draft"].shape, generator=g) < 0.5, d["draft"] % min(V, 97), d["draft"])
    d["pen"] = torch.stack([1 + torch.rand(B, generator=g), torch.rand(B, generator=g) - 0.3, torch.rand(B, generator=g)], 1) \
        * torch.tensor([1.0, 0.125, 1.0])
    if n_bias:
        d["bias_ids"] = torch.randint(-2, V, (B, n_bias), generator=g, dtype=torch.int32)
        d["bias_ids"][:, -1] = d["bias_ids"][:, 0]             # a repeated id: the last entry counts
        d["bias"] = 5 * torch.randn(B, n_bias, generator=g)
    if with_mask:
        d["mask"] = torch.randint(-2 ** 31, 2 ** 31, (B, R, (V + 31) // 32), generator=g).to(torch.int32)
    return x, d


def run(q, x, d, out=None):
    names = {"draft": "draft_tok", "pen": "penalties"}
    kw = {names.get(k, k): v.to(DEV) for k, v in d.items()}
    xg = x.to(DEV)
    out = torch.empty_like(xg) if out is None else xg
    q.qspec_logits_adjust(xg, out, **kw)
    return out


def check(got, x, d):
    want, touched = ref.logits(x, **d)
    got = got.cpu()
    assert torch.equal(got.view(torch.int16)[~touched], x.view(torch.int16)[~touched])
    g64 = got.double()
    assert torch.equal(torch.isinf(g64), torch.isinf(want)) and torch.equal(torch.isnan(g64), torch.isnan(want))
    fin = torch.isfinite(want)
    err = (g64 - want).abs()[fin]
    assert bool((err <= ref.BF16 * want.abs()[fin] + 5 * 64 * 2.0 ** -24).all())


CASES = [(1, 1, 2, 0, 0, False), (1, 4, 40, 5, 3, True), (2, 2, 33, 9, 2, True), (3, 8, 2048, 300, 20, True), (2, 3, 4097, 2000, 7, False),
         (2, 4, 4104, 1024, 0, True), (1, 17, 1000, 50, 9, True), (5, 2, 8192, 0, 4, False), (1, 1, 2055, 1, 1, True)]


@pytest.mark.parametrize("B,R,V,hist,n_bias,with_mask", CASES)
def test_logits(B, R, V, hist, n_bias, with_mask):
    q = lib()
    x, d = inputs(B * 7 + V, B, R, V, hist, n_bias, with_mask)
    out = run(q, x, d)
    q.qspec_check_status()
    check(out, x, d)
    assert torch.equal(run(q, x, d, out="in place").view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("keep", [[], ["pen", "draft"], ["pen", "hist", "hist_len"], ["bias_ids", "bias"], ["mask"],
                                  ["draft"], ["hist", "hist_len"]])
@pytest.mark.parametrize("V", [96, 97])
def test_each_part_alone(keep, V):
    q = lib()
    x, d = inputs(5, 2, 3, V, 40, 6, True)
    d = {k: v for k, v in d.items() if k in keep}
    check(run(q, x, d), x, d)
    q.qspec_check_status()


@pytest.mark.parametrize("V", [64, 65])
def test_infinities_nan_and_rows_without_a_token(V):
    q = lib()
    x, d = inputs(6, 2, 3, V, 30, 5, True)
    x[0, 0, :7] = torch.tensor([float("inf"), float("-inf"), float("nan"), 0.0, -0.0, 3e38, -3e38]).to(torch.bfloat16)
    x[1] = float("-inf")
    d["mask"][0, 1] = 0                                        # a grammar that allows nothing
    d["mask"][0, 0] = -1
    del d["bias_ids"], d["bias"]
    d["pen"][0, 0] = 1.0                                       # (3e38 keeps its size)
    out = run(q, x, d)
    check(out, x, d)
    assert bool((out[0, 1] == float("-inf")).all()) and bool((out[1] == float("-inf")).all())


@pytest.mark.parametrize("V", [2048, 2049])
def test_an_id_many_times_in_the_bias_list(V):
    """The last of many entries of an id counts, at any place in the list, whatever values the others have."""
    q = lib()
    x, d = inputs(11, 2, 3, V, 30, 700, True)
    d["bias_ids"] = d["bias_ids"] % 13 * 150                   # about 54 entries an id, in several ranges of tokens
    special = [float("nan"), 0.0, -0.0, float("inf"), float("-inf"), 2.0 ** -149]
    d["bias"][0, :6] = torch.tensor(special)                   # overruled ones
    d["bias"][1, -6:] = torch.tensor(special)
    d["bias_ids"][1, -6:] = torch.arange(6, dtype=torch.int32) * 150
    out = run(q, x, d)
    q.qspec_check_status()
    check(out, x, d)
    assert torch.equal(run(q, x, d).view(torch.int16), out.view(torch.int16))


def test_long_history_counts():
    """Counts beyond 16 bits, from a history much longer than a block's threads."""
    q = lib()
    n = 70001
    hist = torch.zeros(1, n, dtype=torch.int32)
    hist[0, 1::7] = 5
    x = torch.ones(1, 1, 40).to(torch.bfloat16)
    d = {"hist": hist, "hist_len": torch.tensor([n], dtype=torch.int32), "pen": torch.tensor([[1.0, 2.0 ** -12, 0.25]])}
    out = run(q, x, d)
    q.qspec_check_status()
    check(out, x, d)
    assert float(out[0, 0, 0]) < -10


def test_bad_values_are_reported():
    q = lib()
    base, d0 = inputs(8, 2, 3, 50, 12, 4, False)
    for name, edit in (("draft", lambda t: t.__setitem__((0, 0), 50)), ("draft", lambda t: t.__setitem__((1, 1), -1)),
                       ("hist", lambda t: t.__setitem__((0, 3), 50)), ("hist", lambda t: t.__setitem__((0, 0), -9)),
                       ("hist_len", lambda t: t.__setitem__(1, -1)), ("prompt_len", lambda t: t.__setitem__(0, 13)),
                       ("bias_ids", lambda t: t.__setitem__((1, 2), 50)), ("pen", lambda t: t.__setitem__((1, 0), 0.0))):
        d = {k: v.clone() for k, v in d0.items()}
        edit(d[name])
        out = run(q, base, d)
        with pytest.raises(q.QSpecError, match="INVALID_ARG"):
            q.qspec_check_status()
        q.qspec_check_status()
        if name == "hist_len":
            d["hist_len"][1] = 0
        if name == "prompt_len":                               # (longer than the history: no token was generated)
            pass
        check(out, base, d)
    d = {k: v.clone() for k, v in d0.items()}
    d["hist_len"][0] = 13                                      # more than the row holds: limited to it
    out = run(q, base, d)
    with pytest.raises(q.QSpecError, match="INVALID_ARG"):
        q.qspec_check_status()
    d["hist_len"][0] = 12
    check(out, base, d)


def test_verify_after_adjustment():
    """The adjusted rows through qspec_verify_greedy: a masked draft token is rejected."""
    q = lib()
    B, gamma, V = 1, 3, 1000
    x = torch.zeros(B, gamma + 1, V).to(torch.bfloat16)
    draft = torch.tensor([[10, 20, 30]], dtype=torch.int32)
    for i, t in enumerate((10, 20, 30, 40)):
        x[0, i, t] = 8.0
        x[0, i, 500 + i] = 7.0
    mask = torch.full((B, gamma + 1, (V + 31) // 32), -1, dtype=torch.int32)
    mask[0, 1, 20 // 32] &= ~(1 << 20)
    out = run(q, x, {"mask": mask})
    n, tok = torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(1, gamma + 1, dtype=torch.int32, device=DEV)
    ws = q.new_verify_workspace(B, gamma, V)
    q.qspec_verify_greedy(out, draft.to(DEV), n, tok, ws)
    q.qspec_check_status(ws)
    assert n.tolist() == [1] and tok.tolist() == [[10, 501, -1, -1]]
