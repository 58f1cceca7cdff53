"""Page tables, page copies and compacted tree paths, bit for bit against plain Python written from the definitions."""
import numpy as np
import pytest
import torch

import kv_ref as ref
from gpu_util import DEV, i32_dev, lib

pytestmark = pytest.mark.gpu


def pages_ref(pages, room, parent, keep, need, refs, P, new_width, fill=-5):
    """(table, refs, src, dst, len, left) of qspec_kv_pages; `fill` in the places that are not written."""
    R = len(keep)
    up = lambda n: -(-n // P)  # noqa: E731
    table, refs = [[fill] * new_width for _ in range(R)], list(refs)
    for r in range(R):
        for j in range(up(keep[r])):
            table[r][j] = pages[parent[r]][j]
            refs[table[r][j]] += 1
    for b in range(len(pages)):
        for j in range(up(room[b])):
            refs[pages[b][j]] -= 1
    writer = {}
    for r in range(R):
        if keep[r] % P and need[r] > keep[r]:
            writer.setdefault(table[r][keep[r] // P], []).append(r)
    copies = {r for p, rows in writer.items() for r in (rows[1:] if refs[p] == len(rows) else rows)}
    free = [p for p, c in enumerate(refs) if c == 0]
    lack = sum(up(need[r]) - up(keep[r]) + (r in copies) for r in range(R))
    left = len(free) - lack
    src, dst, size = [-1] * R, [-1] * R, [0] * R
    if left < 0:
        return None, None, src, dst, size, left
    at = iter(free)
    for r in range(R):
        if r in copies:
            j = keep[r] // P
            src[r], dst[r], size[r] = table[r][j], next(at), keep[r] % P
            refs[src[r]] -= 1
            table[r][j] = dst[r]
            refs[dst[r]] = 1
        for j in range(up(keep[r]), up(need[r])):
            table[r][j] = next(at)
            refs[table[r][j]] = 1
    return table, refs, src, dst, size, left


class Step:
    """A table of `rows` rows, some of which share pages, and what the next step wants of it."""

    def __init__(self, seed, rows, new_rows, P, longest, n_free, same=False):
        rng = np.random.default_rng(seed)
        self.P, self.rows, self.new_rows = P, rows, new_rows
        self.width, self.new_width = -(-longest // P) + 1, -(-longest // P) + 3
        self.room = [int(rng.integers(0, longest + 1)) for _ in range(rows)]
        used, self.pages = 0, []
        for b in range(rows):
            n = -(-self.room[b] // P)
            row = []
            if b and rng.random() < 0.5:   # begins with pages of another row
                o = int(rng.integers(0, b))
                row = self.pages[o][:int(rng.integers(0, min(n, -(-self.room[o] // P)) + 1))]
            row = row + list(range(used, used + n - len(row)))
            used = max([used] + [p + 1 for p in row])
            self.pages.append(row + [-99] * (self.width - n))
        self.n_pages = used + n_free
        perm = rng.permutation(self.n_pages).tolist()
        self.pages = [[perm[p] if p >= 0 else p for p in row] for row in self.pages]
        self.refs = [0] * self.n_pages
        for b in range(rows):
            for p in self.pages[b][:-(-self.room[b] // P)]:
                self.refs[p] += 1
        for p in perm[:used // 4]:         # kept by others than the rows
            self.refs[p] += 2
        if same:
            self.parent = list(range(new_rows))
        else:
            self.parent = [int(rng.integers(-1, rows)) if rows else -1 for _ in range(new_rows)]
        self.keep = [int(rng.integers(0, self.room[p] + 1)) if p >= 0 else 0 for p in self.parent]
        self.keep = [self.room[p] if p >= 0 and rng.random() < 0.6 else k for p, k in zip(self.parent, self.keep)]
        self.need = [min(k + int(rng.choice([0, 1, 1, 3, 2 * P])), self.new_width * P) for k in self.keep]

    def expected(self):
        return pages_ref(self.pages, self.room, self.parent, self.keep, self.need, self.refs, self.P, self.new_width)

    def run(self, q, in_place=False, parent=True):
        shape = lambda v, w: i32_dev(np.array(v, dtype=np.int32).reshape(-1, w))  # noqa: E731
        refs = i32_dev(self.refs)
        out = {"table": torch.full((self.new_rows, self.new_width), -5, dtype=torch.int32, device=DEV),
               "refs": refs if in_place else torch.full_like(refs, 77)}
        for n in ("src", "dst", "len"):
            out[n] = torch.full((self.new_rows,), 55, dtype=torch.int32, device=DEV)
        out["left"] = torch.full((1,), 55, dtype=torch.int32, device=DEV)
        q.qspec_kv_pages(shape(self.pages, self.width), i32_dev(self.room), i32_dev(self.keep), i32_dev(self.need), refs, self.P, out["table"],
                         out["refs"], out["src"], out["dst"], out["len"], out["left"], parent=i32_dev(self.parent) if parent else None)
        return {n: t.cpu().tolist() for n, t in out.items()}


@pytest.mark.parametrize("rows,new_rows,P,longest,n_free", [
    (1, 1, 16, 1, 3), (4, 4, 64, 300, 40), (7, 13, 16, 50, 90), (0, 5, 32, 100, 40), (6, 0, 32, 100, 2), (3, 200, 128, 1000, 900),
    (1024, 1024, 16, 90, 9000), (1000, 3, 64, 70, 5), (64, 64, 16, 6000, 20000), (5, 5, 16, 16, 70000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_tables_counts_and_copies(rows, new_rows, P, longest, n_free, in_place):
    q = lib()
    for seed in range(3):
        s = Step(seed, rows, new_rows, P, longest, n_free)
        table, refs, src, dst, size, left = s.expected()
        got = s.run(q, in_place)
        assert got["left"] == [left] and left >= 0
        assert got["src"] == src and got["dst"] == dst and got["len"] == size
        assert got["refs"] == refs and got["table"] == table
        assert sum(refs) == sum(s.refs) - sum(-(-n // P) for n in s.room) + sum(-(-n // P) for n in s.need)
    q.qspec_check_status()


def test_rows_come_from_themselves_without_parents():
    q = lib()
    s = Step(5, 9, 9, 32, 200, 60, same=True)
    table, refs, src, dst, size, left = s.expected()
    got = s.run(q, parent=False)
    assert (got["table"], got["refs"], got["src"], got["dst"], got["len"], got["left"]) == (table, refs, src, dst, size, [left])
    q.qspec_check_status()


@pytest.mark.parametrize("in_place", [False, True])
def test_too_few_pages_change_nothing(in_place):
    q = lib()
    for seed, rows in ((1, 12), (2, 200)):
        s = Step(seed, rows, rows, 16, 60, 0)
        s.need = [s.new_width * s.P] * rows
        left = s.expected()[5]
        got = s.run(q, in_place)
        assert left < 0 and got["left"] == [left] and got["refs"] == s.refs
        assert got["src"] == [-1] * rows and got["dst"] == [-1] * rows and got["len"] == [0] * rows
    q.qspec_check_status()


def test_exactly_enough_pages():
    q = lib()
    for lack in (0, 1):
        s = Step(3, 6, 6, 16, 80, 60)
        s.need = [s.new_width * s.P] * 6   # (more than the old rows release, so that fewer pages are left than were free)
        spare = s.expected()[5]
        free = [p for p, c in enumerate(s.refs) if c == 0]
        for p in free[:spare + lack]:      # taken by someone else
            s.refs[p] = 1
        want = s.expected()
        got = s.run(q)
        assert got["left"] == [want[5]] == [-lack]
        assert got["refs"] == (s.refs if lack else want[1])
    q.qspec_check_status()


def test_bad_numbers_are_reported_and_touch_nothing_else():
    q = lib()
    base = Step(11, 6, 6, 16, 80, 60)
    for change in ("parent", "keep", "need", "room", "id", "count"):
        s = Step(11, 6, 6, 16, 80, 60)
        if change == "parent":
            s.parent[2] = 6
        elif change == "keep":
            s.keep[2], s.need[2] = s.room[s.parent[2]] + 1 if s.parent[2] >= 0 else 1, 80
        elif change == "need":
            s.need[2] = s.new_width * s.P + 1
        elif change == "room":
            s.room[0] = s.width * s.P + 1
        elif change == "id":
            s.pages[[b for b in range(6) if s.room[b]][0]][0] = s.n_pages
        else:
            s.refs[[s.pages[b][0] for b in range(6) if s.room[b]][0]] -= 50
        got = s.run(q)
        with pytest.raises(q.QSpecError, match="QSPEC_ERR_INVALID_ARG"):
            q.qspec_check_status()
        assert len(got["refs"]) == s.n_pages
        if change in ("parent", "keep", "need"):   # that row gets nothing, the others what they would beside an empty row
            s.parent[2], s.keep[2], s.need[2] = -1, 0, 0
            want = s.expected()
            assert (got["table"], got["refs"], got["left"]) == (want[0], want[1], [want[5]])
    got = base.run(q)
    q.qspec_check_status()
    assert got["table"] == base.expected()[0]


def test_steps_in_a_graph_and_on_another_stream():
    """Two steps that swap their buffers, captured once and replayed: pages come and go, and every count comes back."""
    q = lib()
    R, W, P, n = 8, 6, 16, 60
    ends, side = i32_dev([20] * R), torch.cuda.Stream()
    tables = [torch.zeros(R, W, dtype=torch.int32, device=DEV) for _ in range(2)]
    refs = torch.zeros(n, dtype=torch.int32, device=DEV)
    src, dst, size = (torch.zeros(R, dtype=torch.int32, device=DEV) for _ in range(3))
    left, zero = torch.zeros(1, dtype=torch.int32, device=DEV), i32_dev([0] * R)
    none, parent = i32_dev([-1] * R), i32_dev([0, 0, 1, 1, 2, 2, 3, 3])
    q.qspec_kv_pages(tables[1][:0], zero[:0], zero, ends, refs, P, tables[0], refs, src, dst, size, left, parent=none)
    q.qspec_check_status()
    more = i32_dev([21] * R)
    back = i32_dev([20] * R)

    def both():
        q.qspec_kv_pages(tables[0], ends, ends, more, refs, P, tables[1], refs, src, dst, size, left, parent=parent)
        q.qspec_kv_pages(tables[1], more, back, back, refs, P, tables[0], refs, src, dst, size, left)

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for _ in range(5):
        graph.replay()
    q.qspec_check_status()
    table = tables[0].cpu().tolist()
    want = [0] * n
    for row in table:
        for p in row[:2]:
            want[p] += 1
    assert refs.cpu().tolist() == want and left.item() == sum(c == 0 for c in want)
    assert len({row[1] for row in table}) == R # each row writes in a page of its own


@pytest.mark.parametrize("layers,heads,page,dim,n", [(1, 1, 16, 64, 1), (3, 5, 32, 128, 7), (2, 8, 64, 128, 20), (64, 2, 16, 64, 4), (1, 40, 128, 128, 3)])
@pytest.mark.parametrize("part", [False, True])
def test_copies(layers, heads, page, dim, n, part):
    q = lib()
    g = torch.Generator().manual_seed(n + page)
    N = 2 * n + 3
    perm = torch.randperm(N, generator=g).to(torch.int32)
    src, dst = perm[:n].clone(), perm[n:2 * n]
    src[n // 2] = -1 if n > 1 else src[n // 2]
    size = torch.randint(0, page + 1, (n,), generator=g).to(torch.int32)
    size[0] = page
    sets = []
    for _ in range(layers):
        codes = [torch.randint(0, 256, (N, heads, page, dim), generator=g, dtype=torch.uint8) for _ in range(2)]
        exps = [torch.randint(-40, 41, (N, heads), generator=g).to(torch.int8) for _ in range(2)]
        sets.append((codes, exps))
    caches = [q.KVCache(c[0].to(DEV), c[1].to(DEV), e[0].to(DEV), e[1].to(DEV)) for c, e in sets]
    q.qspec_kv_copy_pages(q.KVLayers(caches) if layers > 1 else caches[0], src.to(DEV), dst.to(DEV), lengths=size.to(DEV) if part else None)
    q.qspec_check_status()
    for (codes, exps), cache in zip(sets, caches):
        for c, e, got_c, got_e in zip(codes, exps, (cache.k, cache.v), (cache.k_exp, cache.v_exp)):
            for i in range(n):
                s, d, m = int(src[i]), int(dst[i]), int(size[i]) if part else page
                if s >= 0:
                    c[d, :, :m], e[d] = c[s, :, :m], e[s]
            assert torch.equal(got_c.cpu(), c) and torch.equal(got_e.cpu(), e)


def test_copies_of_bad_pairs_are_reported():
    q = lib()
    cache = q.new_kv_cache(4, 2, 16, 64)
    cache.k.fill_(9)
    cache.k[1].fill_(5)
    before = cache.k.clone()
    for s, d, m in ((4, 0, 16), (1, 4, 16), (1, -1, 16), (1, 0, 17), (1, 0, -1)):
        q.qspec_kv_copy_pages(cache, i32_dev([s]), i32_dev([d]), lengths=i32_dev([m]))
        with pytest.raises(q.QSpecError, match="QSPEC_ERR_INVALID_ARG"):
            q.qspec_check_status()
        assert torch.equal(cache.k, before)


# ---------------------------------------------------------------------------------------- compacting

def compact_ref(bt, nodes, count, first):
    """The path's dequantised values written at the path's positions as the append's definition says."""
    for side in "kv":
        old = [bt.values(side, b) for b in range(bt.B)]
        for b in range(bt.B):
            if not count[b]:
                continue
            base = bt.kv[b] - (bt.tok[b] - first)
            new = old[b][:, base + torch.tensor(nodes[b])]      # [H, count, D]
            for pg in range(base // bt.P, (base + count[b] - 1) // bt.P + 1):
                lo, hi, page = max(base, pg * bt.P), min(base + count[b], (pg + 1) * bt.P), int(bt.table[b, pg])
                for h in range(bt.H):
                    x = new[h, lo - base:hi - base]
                    e, was = ref.block_exp(float(x.abs().max())), int(bt.exps[side][page, h])
                    if lo > pg * bt.P:
                        e = max(e, was)
                        if e > was:                             # every other slot again (NaN codes stay NaN)
                            c = bt.codes[side][page, h]
                            bt.codes[side][page, h] = torch.where((c & 0x7F) == 0x7F, c, ref.e4m3(ref.e4m3_value(c) * 2.0 ** (was - e)))
                    bt.exps[side][page, h] = e
                    bt.codes[side][page, h, lo - pg * bt.P:hi - pg * bt.P] = ref.e4m3(x * 2.0 ** -e)


def path_of(rng, n, count, whole=False):
    return list(range(count)) if whole else sorted(rng.choice(n, count, replace=False).tolist())


@pytest.mark.parametrize("heads,page,dim,nodes,kv,first", [
    (2, 16, 64, [31, 7, 1, 20], [40, 100, 2, 21], 1), (3, 16, 128, [64, 64, 33], [64, 79, 200], 0), (8, 64, 128, [63, 10, 5], [130, 75, 64], 1),
    (9, 32, 64, [40, 2], [41, 35], 1), (1, 128, 128, [64, 12], [129, 128], 2)])
@pytest.mark.parametrize("spread", [0.0, 3.0])
def test_compacted_paths(heads, page, dim, nodes, kv, first, spread):
    q = lib()
    T = max(nodes)
    for seed in range(3):
        rng = np.random.default_rng(seed)
        kv_now = [max(n, m + first) for n, m in zip(kv, nodes)]
        bt = ref.Batch(seed + page, [m + first for m in nodes], kv_now, heads, page, dim, spread=spread)
        cache, batch = bt.gpu(q)
        count = [int(rng.integers(0, n + 1)) if b else n for b, n in enumerate(nodes)]
        path = [path_of(rng, n, c, whole=(b == 0 and seed == 0)) for b, (n, c) in enumerate(zip(nodes, count))]
        table = torch.full((bt.B, T), -1, dtype=torch.int32)
        for b, p in enumerate(path):
            table[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        q.qspec_kv_compact(cache, batch, table.to(DEV), i32_dev(count), first=first)
        q.qspec_check_status()
        compact_ref(bt, path, count, first)
        for side in "kv":
            assert torch.equal(getattr(cache, side + "_exp").cpu(), bt.exps[side])
            assert torch.equal(getattr(cache, side).cpu(), bt.codes[side])


def test_compacting_layers_at_once():
    q = lib()
    bts = [ref.Batch(s, [20, 33], [70, 50], 2, 16, 64) for s in (1, 1, 1)]
    for i, bt in enumerate(bts):
        bt.codes["k"] = torch.where(bt.codes["k"] == 0x7F, bt.codes["k"], (bt.codes["k"] + i) % 0x70)
    pairs = [bt.gpu(q) for bt in bts]
    path = [[1, 4, 9, 10], [0, 31]]
    table = torch.tensor([p + [-1] * (32 - len(p)) for p in path], dtype=torch.int32, device=DEV)
    q.qspec_kv_compact(q.KVLayers([c for c, _ in pairs]), pairs[0][1], table, i32_dev([4, 2]))
    q.qspec_check_status()
    for bt, (cache, _) in zip(bts, pairs):
        compact_ref(bt, path, [4, 2], 1)
        for side in "kv":
            assert torch.equal(getattr(cache, side).cpu(), bt.codes[side]) and torch.equal(getattr(cache, side + "_exp").cpu(), bt.exps[side])


def test_bad_paths_leave_their_sequence_alone():
    q = lib()
    for change in ("node", "negative", "order", "twice", "count", "page", "length", "wide"):
        tok, kv = [9, 9], [40, 40]
        if change == "wide":
            tok, kv = [66, 9], [70, 40]       # 65 nodes
        bt = ref.Batch(2, tok, kv, 2, 16, 64)
        nodes, count = [[0, 3, 7], [2, 5, 6]], [3, 3]
        if change == "node":
            nodes[0][2] = 8
        elif change == "negative":
            nodes[0][0] = -1
        elif change == "order":
            nodes[0] = [3, 0, 7]
        elif change == "twice":
            nodes[0] = [0, 3, 3]
        elif change == "count":
            count[0] = 9
        elif change == "page":
            bt.table[0, 2] = bt.n_pages
        elif change == "length":
            bt.kv[0] = 8
        cache, batch = bt.gpu(q)
        table = torch.full((2, 64), -1, dtype=torch.int32)
        for b in range(2):
            table[b, :3] = torch.tensor(nodes[b], dtype=torch.int32)
        q.qspec_kv_compact(cache, batch, table.to(DEV), i32_dev(count))
        with pytest.raises(q.QSpecError, match="QSPEC_ERR_INVALID_ARG"):
            q.qspec_check_status()
        bt.table[0] = bt.table[1]             # (the reference takes no bad ids; sequence 0 has no path)
        bt.kv[0] = max(bt.kv[0], bt.tok[0])
        compact_ref(bt, [[], nodes[1]], [0, 3], 1)
        for side in "kv":
            assert torch.equal(getattr(cache, side).cpu(), bt.codes[side]) and torch.equal(getattr(cache, side + "_exp").cpu(), bt.exps[side])
