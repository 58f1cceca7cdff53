"""qspec_rotary against the 64-bit rotation.

Tolerance per value: half a bf16 step of the result, and the fp32 part: the angle's sine and cosine are off by
at most 2^-23 (the angle rounded to fp32, one rounding of the result, the factor), the two products and the sum
by 2^-24 each, all relative to |a| + |b|: below 2^-21 (|a| + |b|)."""
import pytest
import torch

import kv_ref as ref
from gpu_util import DEV, lib

pytestmark = pytest.mark.gpu


def check(got, x, pos, w, mult, inter, inverse=False):
    want, size = ref.rotate(x, pos, w, mult, inter, inverse)
    err = (got.double().cpu() - want).abs()
    assert bool((err <= ref.BF16 * want.abs() + 2.0 ** -21 * size).all()), float((err - ref.BF16 * want.abs()).max())


CASES = [  # T, heads, dim, rot, interleaved, scaling, factor
    (1, 1, 8, 2, False, "none", 1.0), (1, 32, 128, 128, False, "none", 1.0), (3, 5, 64, 32, True, "linear", 4.0),
    (17, 3, 72, 40, True, "bands", 8.0), (5, 7, 80, 20, False, "base", 2.0), (5, 2, 80, 20, True, "none", 1.0),
    (9, 4, 128, 96, False, "yarn", 16.0), (33, 40, 128, 96, True, "yarn", 16.0), (2, 3, 48, 6, True, "none", 1.0),
    (1300, 9, 64, 64, False, "bands", 4.0), (5000, 2, 64, 48, False, "none", 1.0), (2, 2, 1024, 1024, False, "none", 1.0)]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("T,H,D,rot,inter,scaling,factor", CASES)
def test_rotary(T, H, D, rot, inter, scaling, factor, inverse):
    q = lib()
    g = torch.Generator().manual_seed(T * 131 + H * 17 + rot)
    x = (3 * torch.randn(T, H, D, generator=g)).to(torch.bfloat16)
    pos = torch.randint(-70000, 1 << 22, (T,), generator=g, dtype=torch.int32)
    pos[0] = 0
    pos[-1] = 2 ** 31 - 1
    kw = dict(original=8192) if scaling in ("bands", "yarn") else {}
    rope = q.Rotary(rot, 500000.0, inter, scaling, factor, **kw)
    w, mult = ref.frequencies(rot, 500000.0, scaling, factor, **kw)
    xg, pg = x.to(DEV), pos.to(DEV)
    out = torch.full_like(xg, 7.0)
    q.qspec_rotary(xg, pg, rope, out, inverse=inverse)
    check(out, x, pos, w, mult, inter, inverse)
    same = xg.clone()
    q.qspec_rotary(same, pg, rope, same, inverse=inverse)      # in place: the same bits
    assert torch.equal(same, out)
    assert torch.equal(out[..., rot:].cpu(), x[..., rot:])


@pytest.mark.parametrize("inter", [False, True])
def test_strides_and_layouts(inter):
    """A [heads, T, dim] input, an output inside a wider buffer, and a broadcast head (stride 0)."""
    q = lib()
    g = torch.Generator().manual_seed(3)
    T, H, D = 7, 5, 64
    pos = torch.arange(100, 100 + T, dtype=torch.int32)
    rope = q.Rotary(48, interleaved=inter)
    w, mult = ref.frequencies(48, 10000.0)
    base = torch.randn(H, T, D, generator=g).to(torch.bfloat16)
    xg = base.to(DEV).transpose(0, 1)
    wide = torch.full((T, 2 * H, D + 8), 5.0, dtype=torch.bfloat16, device=DEV)
    out = wide[:, ::2, :D]
    q.qspec_rotary(xg, pos.to(DEV), rope, out)
    check(out, base.transpose(0, 1), pos, w, mult, inter)
    assert bool((wide[:, 1::2] == 5).all()) and bool((wide[:, :, D:] == 5).all())
    one = base[:1].to(DEV).transpose(0, 1).expand(T, H, D)
    out = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
    q.qspec_rotary(one, pos.to(DEV), rope, out)
    check(out, one.cpu(), pos, w, mult, inter)


def test_inverse_is_the_gradient():
    """<g, R x> = <R^T g, x>, and R^T g against central differences of <g, R x> (fp64 reference, so exact)."""
    q = lib()
    g = torch.Generator().manual_seed(9)
    T, H, D, rot = 3, 2, 32, 24
    pos = torch.tensor([5, 9000, 123456], dtype=torch.int32)
    rope = q.Rotary(rot, scaling="yarn", factor=4.0, original=4096, interleaved=True)
    w, mult = ref.frequencies(rot, 10000.0, "yarn", 4.0, original=4096)
    x, go = (torch.randn(T, H, D, generator=g).to(torch.bfloat16) for _ in range(2))
    gx = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
    q.qspec_rotary(go.to(DEV), pos.to(DEV), rope, gx, inverse=True)
    _, size = ref.rotate(go, pos, w, mult, True, True)
    for t, h, d in [(0, 0, 0), (1, 1, 5), (2, 0, 23), (2, 1, 30)]:
        lo, hi = x.double().clone(), x.double().clone()
        hi[t, h, d] += 0.5
        lo[t, h, d] -= 0.5                     # the map is linear: any step gives the derivative
        num = ((ref.rotate(hi, pos, w, mult, True)[0] - ref.rotate(lo, pos, w, mult, True)[0]) * go.double()).sum()
        assert abs(float(gx[t, h, d]) - float(num)) <= ref.BF16 * abs(float(num)) + 2.0 ** -20 * float(size[t, h, d])


def test_other_stream_and_graph():
    q = lib()
    x = torch.randn(4, 8, 128, device=DEV).to(torch.bfloat16)
    pos = torch.arange(4, dtype=torch.int32, device=DEV)
    rope = q.Rotary(128)
    want, got = torch.empty_like(x), torch.empty_like(x)
    q.qspec_rotary(x, pos, rope, want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    q.qspec_rotary(x, pos, rope, got, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.qspec_rotary(x, pos, rope, got)
    pos += 7
    graph.replay()
    q.qspec_rotary(x, pos, rope, want)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
