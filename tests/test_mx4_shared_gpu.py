"""Attention of requests that share a prefix, on the GPU against the plain 64-bit
forms (bounds: test_mx4_gpu.py; the parts of a row are joined in f32, one more
of the rescalings counted there)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import sparse_attention_lightning_indexer_amd as li  # noqa: E402
from mx4_shared_forms import FORMS, Sizes, lens, of_form, taken  # noqa: E402
from mx4_shared_forms import kind as form_kind  # noqa: E402
from oracle import mx4 as plain  # noqa: E402
from test_mx4_gpu import DEV, Case, check, typed  # noqa: E402


SAMPLE = 8    # rows of a large case compared with the plain form


class Shared(Case):
    """Requests in groups.  The rows of all but a group's first name no page that lies wholly inside the prefix (or,
    hide=False, the first's)."""

    def __init__(self, seed, sizes, kind, hide=True, spread=1.0):
        s = self.sizes = sizes
        rng = self.rng = np.random.default_rng(seed)
        self.lens = np.array(lens(s), dtype=np.int32)
        self.query, self.heads, self.kv, self.d, self.bs, self.kind = s.query, s.heads, s.kv, s.d, s.bs, kind
        self.starts, self.prefixes = list(s.starts), list(s.prefixes)
        self.max_seq_len = max(1, int(self.lens.max()))
        requests, cols = len(self.lens), -(-self.max_seq_len // s.bs)
        shared = np.zeros(requests, dtype=np.int64)          # pages wholly inside the prefix of another's
        first = np.arange(requests)
        for g, prefix in enumerate(self.prefixes):
            for r in range(self.starts[g] + 1, self.starts[g + 1]):
                shared[r], first[r] = max(prefix, 0) // s.bs, self.starts[g]
        self.n_blocks = int((cols - shared).sum()) + 2
        order = rng.permutation(self.n_blocks).astype(np.int32).tolist()
        self.table = np.empty((requests, cols), dtype=np.int32)
        for r in range(requests):
            own = [order.pop() for _ in range(cols - shared[r])]
            self.table[r, shared[r]:] = own
            if shared[r]:
                self.table[r, :shared[r]] = ([-1, 2**31 - 1, self.n_blocks][r % 3] if hide else
                                             self.table[first[r], :shared[r]])
        self.data = [rng.integers(0, 256, (self.n_blocks, s.bs, s.kv, s.d // 2), dtype=np.uint8) for _ in range(2)]
        self.scale = [rng.integers(123, 129, (self.n_blocks, s.bs, s.kv, s.d // 32), dtype=np.uint8) for _ in range(2)]
        self.q_t, self.q = typed(rng.standard_normal((requests * s.query, s.heads, s.d)) * spread, kind)
        self.sm_scale = float(np.float32(1.0 / np.sqrt(s.d)))
        rows = requests * s.query
        self.rows = np.arange(rows)
        if rows > 30 and rows * s.heads * self.max_seq_len > 3e5:     # the first and last row, the last of the first group, some others
            self.rows = np.unique(np.concatenate([[0, rows - 1, self.starts[1] * s.query - 1],
                                                  rng.permutation(rows)[:SAMPLE]]))

    def groups(self):
        on = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
        return dict(prefix_lens=on(self.prefixes), max_prefix_len=max(self.prefixes, default=0),
                    group_starts=on(self.starts),
                    max_group=max((b - a for a, b in zip(self.starts, self.starts[1:])), default=0))

    def want(self, _=None):
        """Of the rows of the sample, from the pages that their requests and groups name."""
        requests = set((self.rows // self.query).tolist())
        requests |= {self.starts[g] for g in range(len(self.prefixes)) for r in list(requests)
                     if self.starts[g] <= r < self.starts[g + 1]}
        table = np.full_like(self.table, -1)
        for r in requests:
            table[r] = self.table[r]
        pages, place = np.unique(np.where((table >= 0) & (table < self.n_blocks), table, 0), return_inverse=True)
        table = np.where((table >= 0) & (table < self.n_blocks), place.reshape(table.shape), -1)
        rows = [plain.values(d[pages], s[pages]) for d, s in zip(self.data, self.scale)]
        return plain.attend_shared(self.q, *rows, table, self.lens, self.query, self.max_seq_len, self.sm_scale,
                                   self.starts, self.prefixes, self.rows)

    def check(self, got, where=""):
        torch.cuda.synchronize()
        out, lse, b = self.want()
        pick = self.rows
        check([x[pick] for x in got], (out[pick], lse[pick], {k: v[pick] for k, v in b.items()}), self.kind, self.d, where)

    def run(self, where="", **kw):
        got = li.mx4_attend_shared(*self.args(), self.max_seq_len, self.sm_scale, **dict(self.groups(), **kw))
        self.check(got, where)
        return got


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("names,d", [(names, d) for names in FORMS for d in FORMS[names]], ids=str)
def test_every_form(names, d, kind):
    """Each form of the two parts at each head dimension, against the plain form; then with NaN in the prefix and in own keys."""
    s = of_form(names, d)
    assert tuple(form_kind(f) for f in taken(s)) == names
    case = Shared(21, s, kind)
    case.run(f"{names} {d}")
    first, last = case.starts[0], len(case.lens) - 1
    for which, head, request, p, block in ((1, 0, first, s.prefixes[0] // 2, 0), (0, s.kv - 1, first, 1, d // 32 - 1),
                                           (1, s.kv - 1, last, int(case.lens[last]) - 1, d // 32 - 1)):
        case.scale[which][case.table[request, p // s.bs], p % s.bs, head, block] = 255
    out, _ = case.run(f"{names} {d} NaN")
    assert torch.isnan(out[:s.query]).any()


@pytest.mark.parametrize("names,d,kind", [
    (("one", "one"), 128, "f16"), (("one+", "one"), 64, "bf16"), (("one+", "pairs"), 96, "f16"), (("two", "one"), 128, "bf16"),
    (("two", "pairs"), 64, "f16"), (("two+", "one"), 192, "bf16"), (("two+", "two"), 128, "f16"), (("two+", "two+"), 256, "f16"),
    (("two+", "one+"), 192, "f16"), (("prompt", "one"), 96, "f16"), (("prompt", "prompt"), 128, "bf16"),
    (("prompt+", "one"), 128, "f16"), (("prompt+", "prompt+"), 96, "bf16"), (("ahead", "one"), 128, "f16"),
    (("ahead+", "one"), 64, "f16")], ids=str)
def test_requests_that_end_inside_the_prefix(names, d, kind):
    """With the prefix in a part of its own: requests that end inside it, that hold fewer keys than they have query rows
    or none, and a first and a last one that are of no group."""
    s = of_form(names, d)
    rng, last = np.random.default_rng(41), len(s.own) - 1
    starts = [min(max(x, 1), last) for x in s.starts]
    own = list(s.own)
    for g, prefix in enumerate(s.prefixes):
        for r in range(starts[g], starts[g + 1]):
            if r % 3 == 1:
                own[r] = -int(rng.integers(1, prefix))
            elif r % 7 == 3:
                own[r] = -prefix + int(rng.integers(1, s.query + 1))
    own[0], own[last] = 40, max(s.query, 33)
    s = s._replace(starts=starts, own=own)
    assert form_kind(taken(s)[0]) != "none"
    case = Shared(42, s, kind)
    case.rows = np.unique(np.concatenate([case.rows, rng.integers(0, (last + 1) * s.query, 20)]))
    case.run(f"{names} {d}")


SHAPES = [
    Sizes([0, 1], [1], [1], 1, 1, 1, 64, 1),
    Sizes([0, 3], [40], [1, 7, 30], 1, 8, 8, 128, 16),
    Sizes([0, 4], [33], [2, 0, 5, 64], 2, 16, 2, 128, 16),
    Sizes([0, 2], [200], [9, 1], 1, 7, 1, 96, 5),
    Sizes([0, 1, 4], [64, 31], [65, 3, 40, 20], 3, 12, 4, 64, 64),
    Sizes([0, 2, 2, 5], [100, 70, 3], [10, 5, 33, 0, 257], 4, 16, 4, 192, 33),
    Sizes([0, 3], [90], [3, 60, 61], 3, 34, 2, 256, 32),
    Sizes([0, 5], [500], [1, 2, 3, 4, 5], 1, 64, 1, 128, 100),
    Sizes([0, 2], [700], [40, 1], 5, 24, 8, 128, 16),
    Sizes([0, 9], [257], [1] * 9, 1, 8, 1, 64, 32),
    Sizes([0, 6], [300], [50, 70, 64, 80, 64, 51], 50, 32, 8, 128, 16),
]


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s.prefixes}x{len(s.own)}q{s.query}d{s.d}")
def test_shared(shape, kind):
    Shared(1, shape, kind).run(f"{shape} {kind}")


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("requests,query,prefix,heads,kv,bs", [
    (3, 1, 2100, 8, 2, 16), (17, 1, 1300, 16, 2, 64), (40, 2, 333, 16, 2, 32), (70, 1, 600, 8, 2, 16),
])
def test_every_head_dimension(requests, query, prefix, heads, kv, bs, d, kind):
    rng = np.random.default_rng(d + requests)
    own = rng.integers(query, 70, requests).tolist()
    own[0], own[-1] = 0, 64
    Shared(2, Sizes([0, requests], [prefix], own, query, heads, kv, d, bs), kind).run(f"{requests} {prefix} {d} {kind}")


def test_groups_of_every_size():
    """Prefixes of none to many keys, around the kernels' steps; groups of none, one and many requests."""
    for seed, prefixes in enumerate(([0, 1, 31, 32, 33], [63, 64, 65, 127, 5], [128, 129, 0, 256, 250])):
        s = Sizes([0, 1, 1, 4, 9, 16], prefixes, [3, 40, 1, 0, 9, 33, 64, 65, 2, 8, 1, 7, 31, 32, 100, 11], 2, 8, 2, 64, 16)
        Shared(seed + 10, s, "f16").run(str(prefixes))


def test_requests_of_no_group():
    """Requests before the first start and behind the last one read all their keys themselves."""
    s = Sizes([2, 4, 5], [70, 40], [50, 3, 6, 9, 12, 33, 80], 2, 8, 2, 128, 16)
    case = Shared(3, s, "bf16")
    assert case.lens.tolist() == [50, 3, 76, 79, 52, 33, 80]
    case.run("no group")
    case.starts = [0, 0, 0]
    case.table = np.where((case.table < 0) | (case.table >= case.n_blocks), 1, case.table)
    case.run("no groups at all", max_group=0)
    case.prefixes, case.starts = [], [0]
    case.run("an empty list of groups", max_group=0)


def test_one_group_without_starts():
    s = Sizes([0, 5], [130], [1, 40, 7, 0, 65], 1, 16, 4, 128, 16)
    case = Shared(4, s, "f16")
    a = case.run("starts")
    b = case.run("no starts", group_starts=None, max_group=None)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_rows_that_see_less_than_the_prefix():
    """Requests shorter than their prefix, lengths of none, more queries than keys, and max_seq_len inside the prefix."""
    s = Sizes([0, 6], [100], [1] * 6, 4, 8, 2, 64, 16)
    case = Shared(5, s, "f16")
    case.lens = np.array([100, 3, 0, 64, 101, 2], dtype=np.int32)
    out, lse = case.run("short")
    assert (out[8:12] == 0).all() and torch.isneginf(lse[8:12]).all() and torch.isneginf(lse[4]).all()
    case.max_seq_len = 70
    case.run("cut")
    case.prefixes = [-5]
    case.table = np.where((case.table < 0) | (case.table >= case.n_blocks), 1, case.table)
    case.run("a negative prefix", max_prefix_len=70)
    case.prefixes = [90]
    want = Shared.want(case)
    case.prefixes = [2**31 - 1]          # counts as max_prefix_len
    got = li.mx4_attend_shared(*case.args(), case.max_seq_len, case.sm_scale, **dict(case.groups(), max_prefix_len=90))
    torch.cuda.synchronize()
    check(got, want, "f16", 64, "a prefix past its limit")


def test_bad_pages():
    """Pages outside the cache hide their keys: of the prefix for all, of own keys for one."""
    s = Sizes([0, 4], [120], [50, 60, 3, 0], 1, 16, 2, 128, 16)
    case = Shared(6, s, "bf16")
    case.table[0, 2], case.table[0, 5], case.table[1, 8:] = -1, case.n_blocks, 2**31 - 1
    case.run("bad pages")
    case.table[0, :] = -7
    case.table[:, 7] = -1
    out, lse = case.run("nothing but bad pages")
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all() and torch.isneginf(lse[2]).all() is not None


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("requests,query,heads,kv", [(5, 2, 8, 2), (40, 1, 64, 8), (64, 4, 64, 8)])
def test_nan_stays_with_the_rows_that_see_it(requests, query, heads, kv, kind):
    """NaN and wild bytes where no row may look; NaN in the prefix for the rows that see it, in own keys for one request."""
    rng = np.random.default_rng(7)
    own = rng.integers(query, 40, requests).tolist()
    s = Sizes([0, requests // 2, requests], [77, 130], own, query, heads, kv, 128, 16)
    case = Shared(7, s, kind)
    used = np.zeros((case.n_blocks, 16), dtype=bool)
    for r in range(requests):
        g = 0 if r < case.starts[1] else 1
        for p in range(int(case.lens[r])):
            used[case.table[case.starts[g] if p < case.prefixes[g] else r, p // 16], p % 16] = True
    for scale in case.scale:
        scale[~used] = 255
    out, lse = case.run("NaN where none looks")
    assert torch.isfinite(out).all()
    first = case.starts[1]
    # the last key of the second request: its last query alone sees it (its own key)
    last = int(case.lens[1]) - 1
    case.scale[1][case.table[1, last // 16], last % 16, 1, 2] = 255
    # a request that ends inside its group's prefix does not see the prefix's last key
    case.lens[first + 1] = 100
    case.scale[1][case.table[first, 120 // 16], 120 % 16, 0, 1] = 255
    case.scale[0][case.table[first, 101 // 16], 101 % 16, kv - 1, 0] = 255
    out, lse = case.run("NaN for some")
    nan_rows = torch.isnan(out).flatten(1).any(1)
    assert nan_rows[2 * query - 1] and not nan_rows[:2 * query - 1].any() and not nan_rows[2 * query:first * query].any()
    short = slice((first + 1) * query, (first + 2) * query)
    assert not nan_rows[short].any() and nan_rows[first * query:(first + 1) * query].all()


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_far_scores_and_small_weights(kind):
    """Scores far from zero on both sides of the prefix's end, and a key of one part that leads all of the other's."""
    s = Sizes([0, 20], [300], [33] * 20, 1, 8, 1, 128, 16)
    case = Shared(8, s, kind, spread=40.0)
    case.run("spread")
    case.sm_scale = float(np.float32(3e4))
    case.run("far")
    case = Shared(9, s, kind)
    case.scale[0][case.table[0, 3], 5] = 134            # one large key in the prefix
    case.run("one key leads")


@pytest.mark.parametrize("order", ["hnd", "scales together"])
def test_other_layouts(order):
    s = Sizes([0, 30], [260], [20] * 30, 1, 32, 4, 128, 16)
    case = Shared(11, s, "f16")
    q, kd, ks, vd, vs, *rest = case.args()
    if order == "hnd":
        kd, ks, vd, vs = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (kd, ks, vd, vs))
    else:
        both = torch.stack((ks, vs), 2)
        ks, vs = both[:, :, 0], both[:, :, 1]
    got = li.mx4_attend_shared(q, kd, ks, vd, vs, *rest, case.max_seq_len, case.sm_scale, **case.groups())
    case.check(got, order)


def test_given_outputs_and_no_lse():
    """Strided outputs, no lse, a workspace of the caller's; nothing else is written."""
    s = of_form(("two+", "one"), 64)
    case = Shared(12, s, "bf16")
    want, requests = case.run(), len(s.own)
    room = torch.full((requests * s.query, s.heads + 1, 80), 5.0, dtype=torch.bfloat16, device=DEV)
    need = li.mx4_attend_shared_workspace_bytes(requests, s.query, case.max_seq_len, 1, requests, max(s.prefixes), s.heads,
                                                s.kv, 64)
    assert need > 0
    workspace = torch.zeros(need + 256, dtype=torch.uint8, device=DEV)
    out, lse = li.mx4_attend_shared(*case.args(), case.max_seq_len, case.sm_scale, **case.groups(), out=room[:, 1:, 8:72],
                                    with_lse=False, workspace=workspace)
    assert lse is None and torch.equal(out, want[0]) and (workspace[need:] == 0).all()
    assert (room[:, 0] == 5).all() and (room[:, :, :8] == 5).all() and (room[:, :, 72:] == 5).all()
    with pytest.raises(li.IndexerError, match="workspace"):
        li.mx4_attend_shared(*case.args(), case.max_seq_len, case.sm_scale, **case.groups(), workspace=workspace[:need - 1])


def test_agrees_with_attention_of_its_own():
    """Tables that name the same pages: the window form's result, within both bounds; and the same bits every time."""
    s = Sizes([0, 32], [1000], [17] * 32, 1, 64, 8, 128, 64)
    case = Shared(13, s, "f16", hide=False)
    full = 1000 // 64
    for a in (*case.data, *case.scale):
        for r in range(1, 32):
            a[case.table[r, full], :1000 % 64] = a[case.table[0, full], :1000 % 64]
    out, lse = case.run()
    case.check(li.mx4_attend_window(*case.args(), case.max_seq_len, case.sm_scale), "alone")
    for _ in range(3):
        again = li.mx4_attend_shared(*case.args(), case.max_seq_len, case.sm_scale, **case.groups())
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("requests,query,prefix,kind", [(40, 1, 2000, "f16"), (3, 70, 500, "bf16"), (5, 2, 60, "f16"),
                                                        (9, 1, 3000, "bf16")])
def test_rows_of_infinities_and_nan_stay_alone(requests, query, prefix, kind):
    """Query rows that hold a NaN, an infinity or the type's largest values: NaN and finite results where attention
    without shared prefixes has them, all other rows as without such rows, within the bounds of the plain form (rows of
    a wave take a new reference for their weights together, so their roundings may differ)."""
    s = Sizes([0, requests], [prefix], [query + i % 5 for i in range(requests)], query, 16, 2, 128, 32)
    case = Shared(31, s, kind, hide=False)
    full = prefix // 32
    for a in (*case.data, *case.scale):
        for r in range(1, requests):
            a[case.table[r, full], :prefix % 32] = a[case.table[0, full], :prefix % 32]
    rest, rest_lse = case.run("plain rows")
    rows = requests * query
    odd = {0: (3, float("nan")), 1: (17, float("inf")), 2: (0, float("-inf")), rows - 2: (9, 0.0), rows - 1: (5, None)}
    for row, (head, value) in odd.items():
        if value is None:
            case.q_t[row, head] = torch.finfo(case.q_t.dtype).max
        else:
            case.q_t[row, head % 16, 7] = value
    out, lse = li.mx4_attend_shared(*case.args(), case.max_seq_len, case.sm_scale, **case.groups())
    alone, alone_lse = li.mx4_attend_window(*case.args(), case.max_seq_len, case.sm_scale)
    assert torch.equal(out.isnan(), alone.isnan()) and torch.equal(lse.isnan(), alone_lse.isnan())
    assert out[0, 3].isnan().all()
    for row, (head, _) in odd.items():
        out[row, head % 16], lse[row, head % 16] = rest[row, head % 16], rest_lse[row, head % 16]
    assert out.isfinite().all() and lse.isfinite().all()
    case.check((out, lse), "beside odd rows")


def test_requests_that_share_little_beside_long_prefixes():
    """A group of a long prefix with one of a short prefix and many own keys, and lone requests: far more own keys
    than the call's sizes say."""
    Shared(32, Sizes([0, 3, 5, 6], [4000, 40, 0], [3, 1, 20, 3900, 2000, 4010], 1, 16, 2, 128, 64), "f16").run()
    Shared(33, Sizes([0, 2, 4], [900, 0], [70, 64, 900, 33], 30, 16, 2, 64, 16), "bf16").run()


def test_streams_and_graphs():
    """Captured calls of their own workspaces replayed side by side, lengths changing between replays."""
    small, large = Sizes([0, 5, 12], [200, 90], [9] * 12, 1, 16, 2, 128, 16), of_form(("two+", "one"), 128)
    cases = [Shared(14, small, "f16"), Shared(15, large, "bf16"), Shared(16, large, "f16")]
    for case in cases:      # pages that leave the prefix become each request's own
        case.table = np.where((case.table < 0) | (case.table >= case.n_blocks), 2, case.table).astype(np.int32)
    streams = [torch.cuda.Stream() for _ in cases]
    held = []
    for case, stream in zip(cases, streams):
        args, groups = case.args(), case.groups()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            out = li.mx4_attend_shared(*args, case.max_seq_len, case.sm_scale, **groups)
        held.append((args, groups, graph, out))
    for step in range(4):
        for case, (args, groups, _, _) in zip(cases, held):
            case.lens = np.maximum(case.lens - step, 0).astype(np.int32)
            case.prefixes = [p - 3 * step for p in case.prefixes]
            args[6].copy_(torch.from_numpy(case.lens))
            groups["prefix_lens"].copy_(torch.tensor(case.prefixes, dtype=torch.int32))
        torch.cuda.synchronize()
        for (_, _, graph, _), stream in zip(held, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for case, (_, _, _, out) in zip(cases, held):
            case.check(out, f"replay {step}")


def test_refusals():
    s = Sizes([0, 4], [90], [3, 20, 1, 33], 2, 8, 2, 64, 16)
    case = Shared(16, s, "f16")
    args, more, groups = case.args(), (case.max_seq_len, case.sm_scale), case.groups()
    lens_ = groups["prefix_lens"]
    for error, change in [
        (TypeError, dict(prefix_lens=lens_.long())),
        (ValueError, dict(prefix_lens=lens_.cpu())),
        (ValueError, dict(group_starts=groups["group_starts"][:1])),
        (ValueError, dict(prefix_lens=lens_.repeat(2), group_starts=None)),
        (ValueError, dict(max_group=5)),
        (ValueError, dict(max_group=-1)),
        (ValueError, dict(max_prefix_len=-1)),
        (ValueError, dict(max_prefix_len=2**32 + 5)),
    ]:
        with pytest.raises(error):
            li.mx4_attend_shared(*args, *more, **dict(groups, **change))
    out, lse = li.mx4_attend_shared(args[0][:0], *args[1:5], args[5][:0], args[6][:0], 2, 64, 0.1, lens_, 90)
    assert out.shape == (0, 8, 64) and lse.shape == (0, 8)


def test_a_server_s_step():
    """Prompt cached, forked, grown, its new tokens normed, rotated and written, and attended with the prompt shared:
    against attention of each request by itself."""
    rng = np.random.default_rng(17)
    bs, kv, heads, d, n_pages, rows, cols, prompt = 16, 2, 8, 128, 120, 12, 12, 100
    kd, vd = (torch.zeros((n_pages, bs, kv, d // 2), dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.full((n_pages, bs, kv, d // 32), 127, dtype=torch.uint8, device=DEV) for _ in range(2))
    pages = li.PageSet([kd, ks, vd, vs])
    refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    table = torch.full((rows, cols), -1, dtype=torch.int32, device=DEV)
    lens_ = torch.zeros(rows, dtype=torch.int32, device=DEV)
    inv = torch.pow(10000.0, -torch.arange(d // 2, device=DEV) / (d // 2)).float()
    weight = torch.rand(d, device=DEV) + 0.5

    def tokens(n, at):
        q, k = (torch.from_numpy(rng.standard_normal((n, h, d))).to(DEV).bfloat16() for h in (heads, kv))
        v = torch.from_numpy(rng.standard_normal((n, kv, d))).to(DEV).bfloat16()
        return (*li.norm_rope(q, k, at, inv, weight, weight), v)

    row = lambda *r: torch.tensor(r, dtype=torch.int32, device=DEV)  # noqa: E731
    slots = li.pages_grow(refs, table, lens_, row(0), prompt, bs)
    _, k, v = tokens(prompt, torch.arange(prompt, device=DEV))
    li.mx4_cache_write(k, slots.view(-1), kd, ks, v, vd, vs)
    children = row(*range(1, 9))
    fresh = li.pages_fork(pages, refs, table, lens_, row(*[0] * 8), children, bs)
    assert (fresh >= 0).all()
    for step in range(20):
        at = lens_[1:9].long()
        slots = li.pages_grow(refs, table, lens_, children, 1, bs)
        q, k, v = tokens(8, at)
        li.mx4_cache_write(k, slots.view(-1), kd, ks, v, vd, vs)
        out, lse = li.mx4_attend_shared(q, kd, ks, vd, vs, table[1:9], lens_[1:9], 1, cols * bs, d**-0.5,
                                        row(prompt), prompt)
        got = [t.cpu().numpy() for t in (kd, ks, vd, vs)]
        rows_ = [plain.values(got[0], got[1]), plain.values(got[2], got[3])]
        want = plain.attend_rows(q.double().cpu().numpy(), *rows_, table[1:9].cpu().numpy(), lens_[1:9].cpu().numpy(), 1,
                                 cols * bs, float(np.float32(d**-0.5)), lambda t, v, e: range(e))
        check((out, lse), want, "bf16", d, f"step {step}")
        if step == 10:      # half the samples end, and the pool moves together
            li.pages_free(refs, table, lens_, row(2, 4, 6, 8))
            place, live = li.pages_compact(pages, refs, table)
            assert live.item() == (refs > 0).sum().item() and (table.max() < live).all()
            li.pages_fork(pages, refs, table, lens_, row(*[0] * 4), row(2, 4, 6, 8), bs)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("names,d", [(("one+", "one"), 128), (("prompt+", "one"), 128), (("none", "ahead"), 64),
                                     (("two+", "two"), 192), (("prompt+", "prompt+"), 96)], ids=str)
def test_requests_whose_pages_are_all_gone(names, d, kind):
    """Requests that name no page of the cache, one of them of no group, beside ones that do: outputs of exactly 0 and
    lse of -inf, finite ones where some key is left; then with the prefix's pages gone, where own keys are all there is."""
    s = of_form(names, d)
    starts = list(s.starts)
    starts[0] = 1                                   # the first request shares nothing
    s = s._replace(starts=starts, own=[max(s.query, 40)] + list(s.own[1:]))
    case = Shared(51, s, kind)
    gone, requests = [0, 3], len(s.own)
    if s.starts[1] < requests - 1:
        gone.append(s.starts[1])                    # the first of another group or of none
    first = {r: s.starts[g] for g in range(len(s.prefixes)) for r in range(s.starts[g], s.starts[g + 1])}
    for r in gone:
        case.table[r] = (-1, case.n_blocks, 2**31 - 1)[r % 3]
    case.rows = np.unique(np.concatenate([case.rows] + [np.arange(r * s.query, r * s.query + min(s.query, 4)) for r in gone]))

    def dead(out, lse, which):
        for r in which:
            at = slice(r * s.query, (r + 1) * s.query)
            assert (out[at] == 0).all() and torch.isneginf(lse[at]).all(), r
    out, lse = case.run(f"{names} {d} some gone")
    dead(out, lse, [r for r in gone if first.get(r, r) in gone])
    assert torch.isfinite(lse[s.query]).all()
    case.table[1] = -5                              # the first group's prefix, and what its first request has of its own
    out, lse = case.run(f"{names} {d} prefix gone")
    dead(out, lse, [r for r in gone + [1] if first.get(r, r) in gone + [1]])


def test_the_most_requests_of_a_group_left_out():
    """max_group None lays several groups out for all requests; with one group of all it is not used, whatever it is."""
    case = Shared(52, Sizes([0, 3, 4, 9], [700, 33, 300], [9, 0, 40, 64, 5, 33, 7, 8, 1], 1, 16, 2, 128, 16), "bf16")
    case.run("several groups", max_group=None)
    case = Shared(53, Sizes([0, 6], [900], [9, 3, 40, 64, 5, 33], 1, 16, 2, 128, 16), "f16")
    a = case.run("all")
    for most in (0, 2, 6):
        b = case.run(f"max_group={most}", group_starts=None, max_group=most)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
