"""What beam selection refuses, before anything reaches a GPU."""
import pytest
import torch

from quantized_speculative_decoding_qspec_gb300 import qspec as q

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    return q.load()


def call(lib, **change):
    a = dict(logits=FAKE, scores=FAKE, done=None, end_tok=0, weights=None, B=2, beams=4, V=1000, n=4, parent=FAKE, tok=FAKE, score=FAKE + 4096,
             ws=FAKE, ws_bytes=1 << 30)
    a.update(change)
    return lib.qspec_beam_select(*a.values(), None)


@pytest.mark.parametrize("change,code", [
    (dict(logits=None), 1), (dict(scores=None), 1), (dict(parent=None), 1), (dict(tok=None), 1), (dict(score=None), 1), (dict(B=0), 1),
    (dict(beams=0), 1), (dict(V=0), 1), (dict(n=0), 1), (dict(n=-1), 1), (dict(beams=33), 2), (dict(n=65), 2), (dict(V=1), 2),
    (dict(V=(1 << 24) + 1), 2), (dict(B=65536), 2), (dict(V=2, beams=1, n=3), 2), (dict(B=65535, beams=32, V=1 << 24), 2),
    (dict(score=FAKE), 1), (dict(score=FAKE + 28), 1), (dict(score=FAKE - 28), 1), (dict(logits=FAKE + 8), 3), (dict(scores=FAKE + 2), 3), (dict(done=FAKE + 1), 3), (dict(weights=FAKE + 2), 3), (dict(tok=FAKE + 2), 3),
    (dict(ws=FAKE + 8), 3), (dict(ws=None), 4), (dict(ws_bytes=65536 * 4), 4)])
def test_arguments(lib, change, code):
    assert call(lib, **change) == code


def test_workspace_sizes(lib):
    assert lib.qspec_beam_workspace_size(0, 4, 1000, 4) == 0 and lib.qspec_beam_workspace_size(1, 33, 1000, 4) == 0
    assert lib.qspec_beam_workspace_size(1, 4, 1000, 65) == 0 and lib.qspec_beam_workspace_size(1, 1, 2, 3) == 0
    small, large = lib.qspec_beam_workspace_size(1, 1, 1000, 1), lib.qspec_beam_workspace_size(64, 8, 152064, 16)
    assert 0 < small < large < 1 << 22 and small > 4 * 65536


def test_the_binding_refuses_short_tensors():
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t)  # noqa: E731
    x, s, f = z(2, 4, 100, t=torch.bfloat16), z(2, 4, t=torch.float32), z(2, 3, t=torch.float32)
    ws = z(64, t=torch.uint8)
    with pytest.raises(ValueError, match="scores holds"):
        q.qspec_beam_select(x, s[:1], z(2, 3), z(2, 3), f, ws)
    with pytest.raises(ValueError, match="tok holds"):
        q.qspec_beam_select(x, s, z(2, 3), z(2, 2), f, ws)
    with pytest.raises(ValueError, match="score holds"):
        q.qspec_beam_select(x, s, z(2, 3), z(2, 3), f[:1], ws)
    with pytest.raises(ValueError, match="done holds"):
        q.qspec_beam_select(x, s, z(2, 3), z(2, 3), f, ws, done=z(7))
    with pytest.raises(ValueError, match="weights holds"):
        q.qspec_beam_select(x, s, z(2, 3), z(2, 3), f, ws, weights=s[:1])
    with pytest.raises(ValueError, match="parent must be"):
        q.qspec_beam_select(x, s, z(3, 3), z(2, 3), f, ws)
    with pytest.raises(TypeError, match="logits must be"):
        q.qspec_beam_select(x.float(), s, z(2, 3), z(2, 3), f, ws)
