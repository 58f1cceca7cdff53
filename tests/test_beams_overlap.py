"""Beam selection and page tables refuse outputs that lie over what they read, or over one another: blocks of one call read while others
write (no GPU)."""
import pytest

from quantized_speculative_decoding_qspec_gb300 import qspec as q

AT = {name: (i + 1) << 24 for i, name in enumerate(
    ["logits", "scores", "done", "weights", "parent", "tok", "score", "ws", "pages", "room", "keep", "need", "refs", "new_pages", "new_refs",
     "src", "dst", "len", "left"])}   # stand-in addresses far apart; never dereferenced


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    return q.load()


def select(lib, **change):
    a = dict(logits=AT["logits"], scores=AT["scores"], done=AT["done"], end_tok=0, weights=AT["weights"], B=3, beams=4, V=1000, n=5,
             parent=AT["parent"], tok=AT["tok"], score=AT["score"], ws=AT["ws"], ws_bytes=1 << 30)
    a.update(change)
    return lib.qspec_beam_select(*a.values(), None)


BEAM_BYTES = {"scores": 48, "done": 48, "weights": 48, "parent": 60, "tok": 60, "score": 60}


@pytest.mark.parametrize("out", ["parent", "tok", "score"])
@pytest.mark.parametrize("other", BEAM_BYTES)
def test_selection(lib, out, other):
    if out == other:
        return
    for at in (AT[other], AT[other] + BEAM_BYTES[other] - 4, AT[other] - BEAM_BYTES[out] + 4):
        assert select(lib, **{out: at}) == 1


def tables(lib, **change):
    a = dict(pages=AT["pages"], room=AT["room"], rows=6, max_pages=8, parent=AT["parent"], keep=AT["keep"], need=AT["need"], new_rows=5,
             new_max_pages=9, refs=AT["refs"], n_pages=100, page=16, new_pages=AT["new_pages"], new_refs=AT["new_refs"], src=AT["src"],
             dst=AT["dst"], len=AT["len"], left=AT["left"])
    a.update(change)
    return lib.qspec_kv_pages(*a.values(), None)


PAGE_IN = {"pages": 192, "room": 24, "parent": 20, "keep": 20, "need": 20, "refs": 400}
PAGE_OUT = {"new_pages": 180, "new_refs": 400, "src": 20, "dst": 20, "len": 20, "left": 4}


@pytest.mark.parametrize("out", PAGE_OUT)
@pytest.mark.parametrize("other", [*PAGE_IN, *PAGE_OUT])
def test_page_tables(lib, out, other):
    if out == other:
        return
    size = {**PAGE_IN, **PAGE_OUT}
    for at in (AT[other], AT[other] + (size[other] - 4) // 16 * 16, AT[other] + 16 - -(-size[out] // 16) * 16):
        if (out, other, at) == ("new_refs", "refs", AT["refs"]):
            continue                     # counts in place
        assert tables(lib, **{out: at}) == 1


def test_counts_in_place_are_read_and_written_alone(lib):
    for out in ("new_pages", "src", "dst", "len", "left"):
        assert tables(lib, new_refs=AT["refs"], **{out: AT["refs"] + 64}) == 1
