"""The page operators on the GPU against the plain forms on lists, bit for bit."""
import copy

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import sparse_attention_lightning_indexer_amd as li  # noqa: E402
from oracle import pages as plain  # noqa: E402

DEV = torch.device("cuda:0")


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Pool:
    """The state on the GPU and on lists."""

    def __init__(self, n_pages, rows, cols, bs, seed=0, shapes=((16, 3, 32), (16, 3, 4), (5,), (16, 24)),
                 dtypes=(torch.uint8, torch.uint8, torch.uint8, torch.float16)):
        self.rng = np.random.default_rng(seed)
        self.bs = bs
        self.gpu = [torch.from_numpy(self.rng.integers(0, 100, (n_pages,) + s)).to(t).to(DEV)
                    for s, t in zip(shapes, dtypes)]
        self.set = li.PageSet(self.gpu)
        self.caches = [t.cpu().numpy() for t in self.gpu]
        self.refs, self.table, self.lens = [0] * n_pages, [[-1] * cols for _ in range(rows)], [0] * rows
        self.g_refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
        self.g_table = torch.full((rows, cols + 3), -1, dtype=torch.int32, device=DEV)[:, :cols]
        self.g_lens = torch.zeros(rows, dtype=torch.int32, device=DEV)

    def put(self):
        """The lists' state onto the GPU."""
        self.g_refs.copy_(ints(self.refs))
        self.g_table.copy_(ints(self.table))
        self.g_lens.copy_(ints(self.lens))

    def same(self, where=""):
        assert self.g_refs.tolist() == self.refs, where
        assert self.g_table.tolist() == self.table, where
        assert self.g_lens.tolist() == self.lens, where
        for a, b in zip(self.gpu, self.caches):
            assert np.array_equal(a.cpu().numpy(), b), where

    def grow(self, rows, tokens, new=None):
        got = li.pages_grow(self.g_refs, self.g_table, self.g_lens, ints(rows), tokens, self.bs,
                            None if new is None else ints(new))
        want = plain.grow(self.refs, self.table, self.lens, rows, tokens, self.bs, new)
        assert got.tolist() == want
        return got

    def fork(self, parents, children):
        got = li.pages_fork(self.set, self.g_refs, self.g_table, self.g_lens, ints(parents), ints(children), self.bs)
        want = plain.fork(self.caches, self.refs, self.table, self.lens, parents, children, self.bs)
        assert got.tolist() == want

    def free(self, rows):
        li.pages_free(self.g_refs, self.g_table, self.g_lens, ints(rows))
        plain.free(self.refs, self.table, self.lens, rows)

    def compact(self):
        place, live = li.pages_compact(self.set, self.g_refs, self.g_table)
        want = plain.compact(self.caches, self.refs, self.table)
        assert place.tolist() == want[0] and live.tolist() == [want[1]]


@pytest.mark.parametrize("n_pages,rows,cols,bs,steps", [
    (60, 12, 9, 4, 60), (7, 5, 4, 3, 40), (300, 40, 30, 1, 30), (400, 9, 300, 16, 30), (2000, 70, 20, 5, 25),
    (1, 2, 2, 2, 10), (20000, 30, 700, 16, 12),
])
def test_a_life_of_requests(n_pages, rows, cols, bs, steps):
    """Random calls one after the other, pools that run out among them; padding and rows named twice in the lists."""
    p = Pool(n_pages, rows, cols, bs, seed=n_pages)
    rng = p.rng

    def some(n, extra=True):
        out = rng.permutation(rows)[:n].tolist()
        if extra and rng.random() < 0.5:
            out += [-1, rows, out[0] if out else -7]
        return out
    for step in range(steps):
        what = rng.integers(0, 5)
        if what == 0:
            tokens = int(rng.integers(1, max(2, cols * bs // 2)))
            members = some(int(rng.integers(1, max(2, rows // 2))))
            new = None if rng.random() < 0.5 else rng.integers(-1, tokens + 2, len(members)).tolist()
            p.grow(members, tokens, new)
        elif what == 1:
            p.grow(some(rows), 1)
        elif what == 2:
            order = rng.permutation(rows).tolist()
            parents, children = order[:max(1, rows // 3)], order[max(1, rows // 3):]
            p.free(children)
            pick = [parents[i] for i in rng.integers(0, len(parents), len(children))]
            if rng.random() < 0.5 and children:
                pick += [rows + 3, parents[0], -1]
                children += [children[0], children[-1], parents[0]]
            p.fork(pick, children)
        elif what == 3:
            p.free(some(int(rng.integers(1, rows))))
        else:
            p.compact()
        p.same((step, int(what)))
    # nothing is lost: without requests every page is free again
    p.free(list(range(rows)))
    p.same()
    assert not any(p.refs)


def test_children_of_one_parent_and_of_several():
    """64 children in any order of three parents, one of whole pages, one empty."""
    p = Pool(500, 70, 40, 8, seed=4)
    p.grow([0, 1, 2], 300, [299, 160, 0])
    p.fork([int(i) for i in p.rng.integers(0, 3, 64)], list(range(3, 67)))
    p.same()
    p.grow(list(range(70)), 9)
    p.same()


def test_long_slots():
    """A prompt's worth of slots, which a second launch writes; rows that cannot grow among them."""
    p = Pool(3000, 5, 900, 16, seed=5)
    p.grow([3, 1, -1, 4, 3], 14000, [14000, 3001, 5, 0, 9])
    p.same()
    p.grow([0, 2, 4], 14397, [14397, 14001, 14400])   # the second finds too few pages
    p.same()


def test_prompts_of_many_pages():
    """Requests that ask for hundreds of pages beside some that ask for one, two, three or none, or find too few."""
    p = Pool(2000, 40, 700, 4, seed=12)
    p.grow([7, 3, 39, 20, 21, 0], 2700, [1, 2699, 8, 9, 0, 2700])
    p.same()
    order = p.rng.permutation(40).tolist()
    p.grow(order + [-1, 40], 1500, [int(v) for v in p.rng.choice([0, 1, 3, 4, 5, 8, 9, 13, 200, 1500], 42)])
    p.same()
    p.free(order[:30])
    p.grow(order, 901)
    p.same()


@pytest.mark.parametrize("tokens", [5, 4000])
def test_a_row_without_its_last_page_does_not_grow(tokens):
    """The partly filled last page is none of the pool's: left as it is; a missing full page before it does not matter."""
    p = Pool(4000, 6, 1100, 8, seed=13)
    p.grow(list(range(6)), 21)
    for row, column, page in ((0, 2, -1), (1, 2, 4000), (2, 2, 2**31 - 1), (3, 1, -7)):
        p.refs[p.table[row][column]] -= 1
        p.table[row][column] = page
    p.put()
    p.grow([0, 1, 2, 3, 4], tokens, [tokens, 0, 4, tokens, tokens])
    p.same()
    assert p.lens[:5] == [21, 21, 21, 21 + tokens, 21 + tokens]


@pytest.mark.parametrize("n_pages", [40000, 16384, 16385])
def test_large_pools(n_pages):
    """More pages than the decision looks at in one step: free ones only far behind, and compaction of all."""
    p = Pool(n_pages, 6, 20, 4, seed=6, shapes=((3,),), dtypes=(torch.uint8,))
    p.refs = [1] * (n_pages - 60) + [0] * 60
    for i in range(0, n_pages - 60, 4001):
        p.refs[i] = 0
    p.put()
    p.grow([0, 1, 2], 70)
    p.fork([0, 0, 1, 2], [3, 4, 4, 5])
    p.same()
    p.refs = [int(r > 0 and p.rng.random() < 0.5) for r in p.refs]   # whatever they were, half of them go
    p.table = [[e if e >= 0 and p.refs[e] else -1 for e in row] for row in p.table]
    p.put()
    p.compact()
    p.same()


def test_copies():
    """Pages in any order; pairs outside the pool or of one page are skipped."""
    p = Pool(50, 1, 1, 4, seed=8)
    order = p.rng.permutation(50).tolist()
    source, target = order[:20] + [-1, 3, 50, 7], order[20:40] + [4, 50, 5, 7]
    target[20] = order[45]
    li.pages_copy(p.set, ints(source), ints(target))
    plain.copy(p.caches, source, target)
    p.same()
    li.pages_copy(p.gpu, ints(source[:1] * 3), ints(order[41:44]))     # one page to several, the caches as a list
    plain.copy(p.caches, source[:1] * 3, order[41:44])
    p.same()


def test_pages_of_any_size_and_place():
    """Pages of 1 to 70001 bytes, strided, at odd addresses, heads before slots; more caches than one launch takes."""
    rng = np.random.default_rng(9)
    n = 30
    tensors = []
    for i, size in enumerate([1, 3, 4, 16, 17, 64, 255, 256, 257, 1024, 4095, 4096, 4097, 16384, 70001] * 6):
        room = torch.from_numpy(rng.integers(0, 256, (n, size + 40)).astype(np.uint8)).to(DEV)
        tensors.append(room[:, (i % 5) * 4 + (i % 3):][:, :size])
    tensors.append(torch.randn((n, 4, 6, 32), device=DEV).half().transpose(1, 2))     # heads before slots
    tensors.append(torch.randn((n, 8), device=DEV)[:, None].double())
    assert len(tensors) > 64
    want = [t.clone() for t in tensors]
    around = [t._base.clone() if t._base is not None else None for t in tensors]
    order = rng.permutation(n)
    a, b = order[:12], order[12:24]
    li.pages_copy(tensors, ints(a.tolist()), ints(b.tolist()))
    at, bt = torch.from_numpy(a).to(DEV), torch.from_numpy(b).to(DEV)
    for t, w in zip(tensors, want):
        w[bt] = w[at]
        assert torch.equal(t, w), t.shape
    # nothing between the pages has moved
    for t, base in zip(tensors[:90], around):
        off = t.storage_offset() % base.shape[1]
        assert torch.equal(t._base[:, :off], base[:, :off])
        assert torch.equal(t._base[:, off + t.shape[1]:], base[:, off + t.shape[1]:])


def test_forks_and_compaction_of_more_caches_than_a_launch_takes():
    p = Pool(90, 9, 12, 4, seed=14, shapes=((4, 5), (4, 2, 16), (33,)) * 25, dtypes=(torch.uint8, torch.float16, torch.uint8) * 25)
    p.grow([0, 1], 46, [46, 13])
    p.fork([0, 1, 1, 0, 0], [2, 3, 4, 5, 8])
    p.same()
    p.grow(list(range(9)), 2)
    p.free([0, 3, 8])
    p.compact()
    p.same()


def test_a_cache_past_2_to_the_32_bytes():
    t = torch.zeros((70, 1 << 26), dtype=torch.uint8, device=DEV)
    t[68, 5], t[69, -1] = 3, 4
    li.pages_copy([t], ints([68, 69]), ints([1, 66]))
    assert int(t[1, 5]) == 3 and int(t[66, -1]) == 4 and int(t.sum(dtype=torch.long)) == 14


def test_bad_entries_are_passed_over():
    """Tables with pages that are not there: never followed, and not handed on."""
    p = Pool(20, 4, 5, 4, seed=10)
    p.grow([0], 14)
    p.table[0][1], p.table[0][3] = 99, 20
    p.table[2] = [-5, 3, 20, -1, -1]
    p.refs[3] += 1
    p.put()
    p.fork([0], [1])
    p.same()
    p.free([2, 0])
    p.same()
    p.table[3] = [77, -9, -1, 2**31 - 1, -2**31]
    p.put()
    p.compact()
    p.same()


def test_no_bytes_and_empty_calls():
    p = Pool(30, 4, 6, 4, seed=11)
    p.grow([0], 9)
    before = [t.clone() for t in p.gpu]
    fresh = li.pages_fork(None, p.g_refs, p.g_table, p.g_lens, ints([0]), ints([2]), p.bs)
    assert fresh.tolist() == plain.fork([], p.refs, p.table, p.lens, [0], [2], p.bs)
    p.free([0])
    place, live = li.pages_compact(None, p.g_refs, p.g_table)
    assert (place.tolist(), live.tolist()[0]) == plain.compact([], p.refs, p.table)
    assert all(torch.equal(a, b) for a, b in zip(p.gpu, before))
    none = ints([])
    li.pages_copy(p.set, none, none)
    li.pages_free(p.g_refs, p.g_table, p.g_lens, none)
    assert li.pages_fork(p.set, p.g_refs, p.g_table, p.g_lens, none, none, 4).shape == (0,)
    assert li.pages_grow(p.g_refs, p.g_table, p.g_lens, none, 3, 4).shape == (0, 3)
    assert li.pages_grow(p.g_refs, p.g_table, p.g_lens, ints([1]), 0, 4).shape == (1, 0)
    p.same()
    # a pool without pages, a table without columns, a table without rows
    empty = torch.empty(0, dtype=torch.int32, device=DEV)
    place, live = li.pages_compact(None, empty, p.g_table.new_empty((0, 4)))
    assert place.shape == (0,) and live.tolist() == [0]
    lens = ints([3, 4])
    li.pages_free(p.g_refs, p.g_table.new_empty((2, 0)), lens, ints([1]))
    assert lens.tolist() == [3, 0]
    lens = ints([3, 0])
    table = ints([[-1, -1], [-1, -1]])
    assert li.pages_grow(empty, table, lens, ints([0, 1]), 1, 4).tolist() == [[-1], [-1]]
    lens = ints([3, 0])
    assert li.pages_fork(None, empty, table, lens, ints([0]), ints([1]), 4).tolist() == [-2]
    assert li.pages_grow(p.g_refs, p.g_table.new_empty((0, 4)), empty, ints([0, -1]), 2, 4).tolist() == [[-1, -1]] * 2


def test_refusals():
    p = Pool(10, 3, 4, 4)
    state = (p.g_refs, p.g_table, p.g_lens)
    rows = ints([0])
    for error, call in [
        (ValueError, lambda: li.PageSet([])),
        (ValueError, lambda: li.PageSet([torch.zeros(4, 4)])),
        (ValueError, lambda: li.PageSet([p.gpu[0], p.gpu[1][:5]])),
        (ValueError, lambda: li.PageSet([p.gpu[0][..., :16]])),
        (ValueError, lambda: li.PageSet([p.gpu[0][:, :0]])),
        (li.IndexerError, lambda: li.pages_copy([torch.zeros(1, 8, device=DEV).expand(9, 8)], rows, rows)),
        (TypeError, lambda: li.pages_copy(p.set, rows.long(), rows)),
        (ValueError, lambda: li.pages_copy(p.set, rows, ints([1, 2]))),
        (ValueError, lambda: li.pages_copy(p.set, rows.cpu(), rows)),
        (ValueError, lambda: li.pages_fork(p.set, p.g_refs[:5], p.g_table, p.g_lens, rows, rows, 4)),
        (ValueError, lambda: li.pages_fork(p.set, *state, rows, ints([1, 2]), 4)),
        (li.IndexerError, lambda: li.pages_fork(p.set, *state, rows, rows, 0)),
        (ValueError, lambda: li.pages_grow(p.g_refs, p.g_table, p.g_lens[:2], rows, 1, 4)),
        (ValueError, lambda: li.pages_grow(*state, rows, -1, 4)),
        (ValueError, lambda: li.pages_grow(*state, rows, 1, 4, ints([1, 2]))),
        (ValueError, lambda: li.pages_grow(*state, rows, 1, 4, slots=torch.zeros((1, 2), dtype=torch.long, device=DEV))),
        (ValueError, lambda: li.pages_free(p.g_refs, p.g_table.t(), p.g_lens, rows)),
        (TypeError, lambda: li.pages_free(p.g_refs.float(), p.g_table, p.g_lens, rows)),
        (ValueError, lambda: li.pages_compact(p.set, p.g_refs, p.g_table, place=ints([1]))),
        (li.IndexerError, lambda: li.pages_compact(p.set, p.g_refs, p.g_table,
                                                   workspace=torch.zeros(8, dtype=torch.uint8, device=DEV))),
    ]:
        with pytest.raises(error):
            call()
    p.same()


def test_a_stream_and_a_graph():
    """A step of a server captured once and replayed: free, fork, grow and compact, with eager calls between."""
    p = Pool(200, 12, 8, 4, seed=12)
    p.grow([0, 1], 27, [27, 13])
    parents, children = [0, 1, 0, 0], [4, 5, 6, 11]
    args = (ints(parents), ints(children))
    fresh, slots = torch.empty(4, dtype=torch.int32, device=DEV), torch.empty((4, 3), dtype=torch.long, device=DEV)
    place, live = torch.empty(200, dtype=torch.int32, device=DEV), torch.empty(1, dtype=torch.int32, device=DEV)
    workspace = torch.empty(li.pages_compact_workspace_bytes(200), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):      # another stream than the tensors' own
        li.pages_fork(p.set, p.g_refs, p.g_table, p.g_lens, *args, p.bs)
    torch.cuda.current_stream().wait_stream(side)
    plain.fork(p.caches, p.refs, p.table, p.lens, parents, children, p.bs)
    p.same()
    state = (p.g_refs, p.g_table, p.g_lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        li.pages_free(*state, args[1])
        li.pages_fork(p.set, *state, *args, p.bs, fresh=fresh)
        li.pages_grow(*state, args[1], 3, p.bs, slots=slots)
        li.pages_compact(p.set, p.g_refs, p.g_table, place, live, workspace)
    for step in range(4):
        p.grow([0, 1, 2], 1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        plain.free(p.refs, p.table, p.lens, children)
        assert fresh.tolist() == plain.fork(p.caches, p.refs, p.table, p.lens, parents, children, p.bs)
        assert slots.tolist() == plain.grow(p.refs, p.table, p.lens, children, 3, p.bs)
        assert (place.tolist(), live.item()) == plain.compact(p.caches, p.refs, p.table)
        p.same(step)


def test_the_same_pages_every_time():
    """What a call does depends on its state alone."""
    p = Pool(800, 64, 30, 4, seed=13)
    p.grow([0, 1, 2], 110, [110, 57, 84])
    start = copy.deepcopy((p.refs, p.table, p.lens))
    results = []
    for _ in range(5):
        p.refs, p.table, p.lens = copy.deepcopy(start)
        p.put()
        p.fork([i % 3 for i in range(50)], list(range(5, 55)))
        p.grow(list(range(64)), 5)
        results.append((p.g_refs.clone(), p.g_table.clone()))
    assert all(torch.equal(a, b) for r in results[1:] for a, b in zip(r, results[0]))


def test_a_child_of_a_row_without_its_last_page_has_none_either():
    """A parent whose partly filled last page is none of the pool's hides its last tokens: the child takes no page, which
    would show them bytes of whoever held it before.  The page of its turn stays free, later children get theirs."""
    p = Pool(60, 40, 6, 4, seed=15, shapes=((4, 3),), dtypes=(torch.uint8,))
    p.grow([0, 1, 2, 3, 4], 18, [18, 18, 18, 16, 2])
    for row, column, page in ((0, 4, -1), (1, 4, 60), (4, 0, -2**31)):
        p.refs[p.table[row][column]] -= 1
        p.table[row][column] = page
    p.put()
    parents = [0, 2, 1, 3, 4, 2, 0, 0, 2, 1, 4]
    got = li.pages_fork(p.set, p.g_refs, p.g_table, p.g_lens, ints(parents), ints(list(range(10, 21))), p.bs).tolist()
    assert [f >= 0 for f in got] == [x == 2 for x in parents] and min(got) == -1
    assert p.g_lens.tolist()[10:21] == [18, 18, 18, 16, 2, 18, 18, 18, 18, 18, 2]
    table = p.g_table.tolist()
    assert all(table[10 + i][4] == -1 for i, x in enumerate(parents) if x in (0, 1)) and table[14] == table[20] == [-1] * 6
    assert got == plain.fork(p.caches, p.refs, p.table, p.lens, parents, list(range(10, 21)), p.bs)
    p.same()
    p.grow(list(range(10, 21)), 1)       # those children do not grow, as their parents would not
    p.same()
    p.free(list(range(40)))
    p.same()
    assert max(p.refs) == 0              # nothing is held without a request


def _long_list(rng, rows, n):
    """Rows in any order, the same row on both sides of each 1024th entry, named again far behind, and padding."""
    out = rng.permutation(rows)[:n].tolist()
    out += [-1] * (n - len(out))
    for at in range(1024, n, 1024):
        out[at] = out[at - 1]
    for at in range(7, n, 97):
        out[at] = (-1, rows, 2**31 - 1, out[at // 2])[at % 4]
    return out


@pytest.mark.parametrize("n", [1023, 1024, 1025, 2500, 8192])
def test_long_lists(n):
    """Lists of more entries than the deciding workgroup looks at in one step, in tables as long as they may be."""
    rows = 8192
    p = Pool(3 * n, rows, 6, 4, seed=n, shapes=((3,), (4, 4)), dtypes=(torch.uint8, torch.float16))
    rng = p.rng
    members = _long_list(rng, rows, n)
    p.grow(members, 24, rng.choice([0, 1, 3, 4, 5, 9], n).tolist())
    p.same("some pages each")
    p.grow(_long_list(rng, rows, n), 1)
    p.same("one token each")
    # parents and children in any order: full pages shared, a copy of the last one
    order = rng.permutation(rows).tolist()
    parents, children = order[:600], order[600:]
    p.free(children)
    p.same("children freed")
    child = _long_list(rng, len(children), n)
    child = [children[c] if 0 <= c < len(children) else c for c in child]
    parent = [parents[i] for i in rng.integers(0, 600, n)]
    for at in range(5, n, 61):
        parent[at] = (-1, rows)[at % 2]
    p.fork(parent, child)
    p.same("forked")
    p.free(_long_list(rng, rows, n))
    p.same("freed")
    p.compact()
    p.same("moved together")


@pytest.mark.parametrize("n,free", [(2500, 1030), (2500, 2047), (8192, 1024), (8192, 5000), (1025, 1024)])
def test_long_lists_that_run_out_of_pages(n, free):
    """The pages end behind the first 1024 entries: of those that grow by one page or by several, and of children."""
    rows = 8192
    p = Pool(free + 300, rows, 5, 4, seed=n + free, shapes=((5,),), dtypes=(torch.uint8,))
    rng = p.rng
    held = sorted(rng.permutation(free + 300)[:300].tolist())
    for page in held:                       # pages in use anywhere in the pool
        p.refs[page] = 1
    p.put()
    p.grow(_long_list(rng, rows, n), 4)
    p.same("a page each")
    p.free(list(range(rows)))
    p.same("none")
    p.grow(_long_list(rng, rows, n), 20, rng.choice([0, 2, 4, 7, 20], n, p=[.3, .5, .1, .05, .05]).tolist())
    p.same("some pages each")
    p.free(list(range(rows)))
    order = rng.permutation(rows).tolist()
    p.grow(order[:3], 7, [7, 4, 6])
    child = [order[3 + c] if 0 <= c < rows - 3 else c for c in _long_list(rng, rows - 3, n)]
    p.fork([order[i] for i in rng.choice(3, n, p=[.45, .1, .45])], child)
    p.same("children")
    p.compact()
    p.same("moved together")
