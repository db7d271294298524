"""The 4-bit cache operators on the GPU against the plain 64-bit forms.

Error bounds of the attention, derived from the arithmetic.  With u the
largest relative error of a rounding to the query's type (2^-11 f16, 2^-8
bf16) and w the exact softmax weights of a row over n keys:
  * q and the cached values are exact in the type, so a score z is off by the
    f32 sum of d exact products, at most 2 d 2^-24 sum|q k| sm_scale (a factor 2
    for the matrix unit's unspecified order and truncation), by the rounding of
    sm_scale * log2 e and of z * log2 e - m (2^-23 (|z| + |m|), m another
    score) and by the exponential's last bit: delta <= d 2^-23 reach + 2^-22 (top + 1)
  * a weight is then off by a factor e^delta, as is their sum: 2 delta together
  * each weight is rounded to the type before the product with V (u), the
    result once more (u |out|), and f32 sums of n terms, the rescalings and
    the final quotient add (n + 64) 2^-23
  out:  (u + 2 delta + (n + 64) 2^-23) sum w|V| + u |out|, and where the type is f16
        the absolute rounding of weights and results below its normal range,
        2^-25 sum|V| + 2^-25 (the largest weight is 1 against the running
        maximum, so the sum the weights are divided by is at least 1);
        for either type 2^-126 (sum|V| + 1): a weight 2^x with x < -126, against the
        largest weight 2^0, is below f32's normal range and the exponential gives 0
        for it, an absolute error under 2^-126 each, with the same sum of at least 1
        below it; for instance scores of 611.5 and 395.9 differ by 311 in powers of
        two, and where the first key's V is 0 the exact result, 9e-95, is below f32
  lse:  delta + (n + 64) 2^-23 + 2^-22 (|lse| + 1)
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import sparse_attention_lightning_indexer_amd as li  # noqa: E402
from oracle import mx4 as plain  # noqa: E402

DEV = torch.device("cuda:0")
DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {"f16": 2.0**-11, "bf16": 2.0**-8}


def typed(x, kind):
    """An f64 array as a CPU tensor of the type, and the f64 values it holds."""
    t = torch.from_numpy(np.asarray(x, dtype=np.float64)).to(DTYPE[kind])
    return t, t.double().numpy()


# ------------------------------------------------------------------ the cache

def fresh(n_blocks, bs, heads, d, order="nhd"):
    """A cache of recognisable bytes, contiguous or as a view of another order."""
    def make(width, fill):
        if order == "nhd":
            return torch.full((n_blocks, bs, heads, width), fill, dtype=torch.uint8, device=DEV)
        if order == "hnd":
            return torch.full((n_blocks, heads, bs, width), fill, dtype=torch.uint8, device=DEV).transpose(1, 2)
        big = torch.full((n_blocks, bs, heads + 1, width + 16), fill, dtype=torch.uint8, device=DEV)   # "padded"
        return big[:, :, 1:, 16:]
    return make(d // 2, 0xA5), make(d // 32, 0x5A)


def check_written(x, slots, data, scale, kind, n_blocks, bs, where):
    """The cache's bytes: written slots hold the plain form's, others their old ones."""
    want_d, want_s = plain.quantise(x, kind)
    got_d, got_s = (t.contiguous().view(-1, *t.shape[2:]).cpu().numpy() for t in (data, scale))
    touched = np.zeros(n_blocks * bs, dtype=bool)
    for t, s in enumerate(slots):
        if 0 <= s < n_blocks * bs:
            touched[s] = True
            assert np.array_equal(got_s[s], want_s[t]), (where, t, s)
            # a block of NaN has codes 0; -0 and +0 are different codes of equal value, and both are pinned
            assert np.array_equal(got_d[s], want_d[t]), (where, t, s)
    assert (got_d[~touched] == 0xA5).all() and (got_s[~touched] == 0x5A).all(), where


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("n,heads,d,bs,order", [
    (1, 1, 32, 1, "nhd"), (1, 8, 128, 64, "nhd"), (5, 3, 96, 7, "nhd"), (33, 2, 64, 16, "hnd"), (17, 5, 160, 3, "padded"),
    (3, 1, 1024, 16, "nhd"), (70, 4, 256, 33, "hnd"), (130, 1, 32, 64, "padded"),
])
def test_write_and_read(kind, n, heads, d, bs, order):
    rng = np.random.default_rng(n * 1000 + d)
    x = [typed(rng.standard_normal((n, heads, d)) * np.exp2(rng.integers(-9, 9, (n, heads, 1))), kind) for _ in range(2)]
    n_blocks = -(-n // bs) + 2
    slots = rng.permutation(n_blocks * bs)[:n].astype(np.int64)
    if n > 3:
        slots[1], slots[3] = -1, n_blocks * bs + 5        # padding, and a slot past the cache
    kd, ks = fresh(n_blocks, bs, heads, d, order)
    vd, vs = fresh(n_blocks, bs, heads, d, order)
    s = torch.from_numpy(slots).to(DEV)
    li.mx4_cache_write(x[0][0].to(DEV), s, kd, ks, x[1][0].to(DEV), vd, vs)
    torch.cuda.synchronize()
    for (t, v), data, scale in zip(x, (kd, vd), (ks, vs)):
        check_written(v, slots, data, scale, kind, n_blocks, bs, f"{kind} {order}")
        got = li.mx4_cache_read(data, scale, s, DTYPE[kind]).double().cpu().numpy()
        want = plain.values(*plain.quantise(v, kind))
        want[(slots < 0) | (slots >= n_blocks * bs)] = 0.0
        assert np.array_equal(got, want)                   # exact: every stored value is of the type


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_write_and_read_many(kind):
    """More values than the caches hold (the streaming forms), against the same rows written a few at a time."""
    n, heads, d = 20011, 7, 128
    x = (torch.randn((n, heads, d), device=DEV) * 3).to(DTYPE[kind])
    slots = torch.randperm(n + 50, device=DEV)[:n]
    slots[::101] = -1
    big, small = fresh(n + 50, 1, heads, d), fresh(n + 50, 1, heads, d)
    li.mx4_cache_write(x, slots, *big)
    for a in range(0, n, 4000):
        li.mx4_cache_write(x[a:a + 4000], slots[a:a + 4000], *small)
    assert all(torch.equal(p, q) for p, q in zip(big, small))
    got = li.mx4_cache_read(*big, slots, DTYPE[kind])
    parts = [li.mx4_cache_read(*small, slots[a:a + 4000], DTYPE[kind]) for a in range(0, n, 4000)]
    assert torch.equal(got, torch.cat(parts)) and (got[::101] == 0).all()
    few = torch.arange(3, 40, device=DEV)
    want = plain.values(*plain.quantise(x[few].double().cpu().numpy(), kind))
    want[slots[few].cpu().numpy() < 0] = 0.0
    assert np.array_equal(got[few].double().cpu().numpy(), want)


def test_write_one_tensor_and_strided_rows():
    """K alone, taken from a fused projection's output, into one cache."""
    rng = np.random.default_rng(2)
    t, _ = typed(rng.standard_normal((9, 3 * 2 * 64)), "f16")
    fused = t.to(DEV)
    k = fused[:, 128:256].view(9, 2, 64)
    kd, ks = fresh(2, 8, 2, 64)
    slots = np.arange(9, dtype=np.int64) + 3
    li.mx4_cache_write(k, torch.from_numpy(slots).to(DEV), kd, ks)
    check_written(k.double().cpu().numpy(), slots, kd, ks, "f16", 2, 8, "strided")


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_every_bit_pattern(kind):
    """Every 16-bit pattern: alone in a block of zeros, among its neighbours, and under a larger value."""
    bits = np.arange(65536, dtype=np.uint16)
    near = bits.reshape(2048, 1, 32)
    alone = np.zeros((65536, 1, 32), dtype=np.uint16)
    alone[:, 0, 7] = bits
    top = near.copy()
    top[:, 0, 0] = {"f16": 0x4480, "bf16": 0x4090}[kind]       # 4.5: the codes' scale is then at least 1
    for name, pattern in (("near", near), ("alone", alone[::3]), ("top", top)):
        t = torch.from_numpy(pattern.astype(np.int16)).view(DTYPE[kind])
        n = len(pattern)
        kd, ks = fresh(-(-n // 64), 64, 1, 32)
        s = torch.arange(n, device=DEV)
        li.mx4_cache_write(t.to(DEV), s, kd, ks)
        check_written(t.double().numpy(), np.arange(n), kd, ks, kind, kd.shape[0], 64, f"{kind} {name}")


def test_read_rounds_once_and_repeats():
    """Every code under every scale, read as either type; the same slot twice; invalid slots read as zeros."""
    d, n = 64, 256
    data = torch.arange(256, dtype=torch.uint8).view(-1, 1).expand(256, 16).repeat(1, 2).view(n, 1, 1, 32).contiguous()
    for s0 in range(256):
        scale = torch.full((n, 1, 1, 2), s0, dtype=torch.uint8)
        scale[:, :, :, 1] = 127
        want = plain.values(data.numpy().reshape(n, 1, 32), scale.numpy().reshape(n, 1, 2))
        slots = torch.cat([torch.arange(n), torch.tensor([5, 5, -3, n, 2**40])])
        for kind in ("f16", "bf16"):
            got = li.mx4_cache_read(data.to(DEV), scale.to(DEV), slots.to(DEV), DTYPE[kind]).cpu()
            ref = torch.from_numpy(want).to(DTYPE[kind])          # rounded from 64 bits, once
            ref = torch.cat([ref, ref[5:6], ref[5:6], torch.zeros_like(ref[:3])])
            assert torch.equal(torch.nan_to_num(got, nan=1.5), torch.nan_to_num(ref, nan=1.5)), (s0, kind)
            assert torch.equal(torch.isnan(got), torch.isnan(ref)), (s0, kind)


def test_read_into_rows_of_a_larger_tensor():
    rng = np.random.default_rng(4)
    data = torch.from_numpy(rng.integers(0, 256, (3, 5, 2, 48), dtype=np.uint8)).to(DEV)
    scale = torch.from_numpy(rng.integers(118, 130, (3, 5, 2, 3), dtype=np.uint8)).to(DEV)
    big = torch.full((4, 2, 112), 7.0, dtype=torch.float16, device=DEV)
    got = li.mx4_cache_read(data, scale, torch.tensor([14, 0, 7, 14], device=DEV), out=big[:, :, 8:104])
    want = plain.values(data.cpu().numpy().reshape(15, 2, 48), scale.cpu().numpy().reshape(15, 2, 3))[[14, 0, 7, 14]]
    assert got.data_ptr() == big[:, :, 8:].data_ptr()
    assert np.array_equal(big[:, :, 8:104].double().cpu().numpy(), want)
    assert (big[:, :, :8] == 7.0).all() and (big[:, :, 104:] == 7.0).all()


# --------------------------------------------------------------- the attention

class Case:
    """A cache of random codes, its pages in a random order, and queries."""

    def __init__(self, seed, lens, query, heads, kv, d, bs, kind, spread=1.0):
        rng = self.rng = np.random.default_rng(seed)
        self.lens = np.array(lens, dtype=np.int32)
        self.query, self.heads, self.kv, self.d, self.bs, self.kind = query, heads, kv, d, bs, kind
        R = len(lens)
        self.max_seq_len = max(1, int(max(lens, default=1)))
        per = -(-self.max_seq_len // bs)
        self.n_blocks = R * per + 2
        self.table = rng.permutation(self.n_blocks)[: R * per].reshape(R, per).astype(np.int32)
        self.data = [rng.integers(0, 256, (self.n_blocks, bs, kv, d // 2), dtype=np.uint8) for _ in range(2)]
        self.scale = [rng.integers(123, 129, (self.n_blocks, bs, kv, d // 32), dtype=np.uint8) for _ in range(2)]
        self.q_t, self.q = typed(rng.standard_normal((R * query, heads, d)) * spread, kind)
        self.sm_scale = float(np.float32(1.0 / np.sqrt(d)))

    def args(self):
        on = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
        return (self.q_t.to(DEV), on(self.data[0]), on(self.scale[0]), on(self.data[1]), on(self.scale[1]),
                on(self.table), on(self.lens), self.query)

    def want(self, positions):
        rows = [plain.values(d, s) for d, s in zip(self.data, self.scale)]
        return plain.attend_rows(self.q, *rows, self.table, self.lens, self.query, self.max_seq_len, self.sm_scale,
                                 positions)

    def seen(self, t):
        r, j = divmod(t, self.query)
        return int(self.lens[r]) - self.query + 1 + j


def check(got, want, kind, d, where):
    out, lse = (x.double().cpu().numpy() for x in got)
    o, l, b = want
    n = b["count"][:, None]
    delta = d * 2.0**-23 * b["reach"] + 2.0**-22 * (b["top"] + 1)
    tol_l = delta + (n + 64) * 2.0**-23 + 2.0**-22 * (np.abs(l) + 1)
    assert np.array_equal(np.isneginf(lse), np.isneginf(l)), where
    assert np.array_equal(np.isnan(lse), np.isnan(l)), where
    fine = np.isfinite(l)
    assert np.all(np.abs(lse - np.where(fine, l, 0))[fine] <= tol_l[fine]), (
        where, float(np.max((np.abs(lse - l) / tol_l)[fine])))
    assert np.array_equal(np.isnan(out), np.isnan(o)), where
    tol = (UNIT[kind] + 2 * delta + (n + 64) * 2.0**-23)[..., None] * b["spread"] + UNIT[kind] * np.abs(o)
    tol = tol + (2.0**-25 if kind == "f16" else 2.0**-126) * (b["plain"] + 1)
    ok = ~np.isnan(o)
    err = np.abs(out - np.where(ok, o, 0))
    bad = ok & (err > tol)
    assert not bad.any(), (where, np.argwhere(bad)[:4].tolist(), float(np.max((err / (tol + 1e-300))[ok])))


def selection(case, k, pool=1, holes=0.1):
    """Distinct entries of each row's visible units in random order, some of them -1, -1 behind the last."""
    rows = case.q.shape[0]
    idx = np.full((rows, k), -1, dtype=np.int32)
    for t in range(rows):
        units = -(-max(case.seen(t), 0) // pool)
        pick = case.rng.permutation(units)[:k]
        idx[t, : len(pick)] = pick
        idx[t, case.rng.random(k) < holes] = -1
    return idx


def run_selected(case, idx, pool=1, where="", **kw):
    got = li.mx4_attend_selected(*case.args(), torch.from_numpy(idx).to(DEV), case.sm_scale, pool_size=pool, **kw)
    torch.cuda.synchronize()
    want = case.want(lambda t, v, e: plain.positions_selected(idx[t], pool, e))
    check(got, want, case.kind, case.d, where)
    return got


def run_window(case, window, sinks, where="", **kw):
    got = li.mx4_attend_window(*case.args(), case.max_seq_len, case.sm_scale, window=window, sinks=sinks, **kw)
    torch.cuda.synchronize()
    want = case.want(lambda t, v, e: plain.positions_window(v, e, window, sinks))
    check(got, want, case.kind, case.d, where)
    return got


# (lens, query, heads, kv heads, d, block size)
SHAPES = [
    ([1], 1, 1, 1, 64, 1),
    ([1, 0, 2], 1, 8, 8, 128, 16),
    ([31, 32, 33], 1, 16, 2, 128, 16),
    ([200], 1, 7, 1, 96, 5),
    ([65, 300], 2, 12, 4, 64, 64),
    ([100, 3, 0, 257], 4, 16, 4, 192, 33),
    ([90, 150], 3, 34, 2, 256, 32),
    ([500], 1, 64, 1, 128, 100),
    ([700, 40], 5, 24, 8, 128, 16),
]


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("k", [1, 31, 96, 333])
def test_selected(shape, k, kind):
    case = Case(7, *shape, kind)
    run_selected(case, selection(case, k), where=f"{shape} {k} {kind}")


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (33, 4), (64, 70), (129, 1), (5000, 3)])
def test_window(shape, window, sinks, kind):
    case = Case(8, *shape, kind)
    run_window(case, window, sinks, where=f"{shape} {window}+{sinks} {kind}")


@pytest.mark.parametrize("pool", [2, 5, 16, 32, 100])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_selected_pools(pool, kind):
    case = Case(9, [311, 1, 64, 33], 2, 8, 2, 128, 16, kind)
    run_selected(case, selection(case, 9, pool), pool, where=f"pool {pool} {kind}")


def test_selected_entries_out_of_sight():
    """Indices past the visible keys, past the table, negative, huge and twice the same."""
    case = Case(10, [50, 20], 2, 8, 2, 64, 16, "f16")
    idx = np.array([[0, 49, 48, 60, -5, 2**31 - 1, 3, 3], [49, 50, -2**31, 1, 63, 64, 7, 8],
                    [-1] * 8, [19, 19, 19, 20, 21, 0, -1, 1 << 30]], dtype=np.int32)
    run_selected(case, idx, where="out of sight")
    idx = np.where(idx >= 0, idx // 3, idx)
    run_selected(case, idx.astype(np.int32), 3, where="out of sight, pooled")


def test_empty_selections_and_rows():
    case = Case(11, [9, 0], 1, 4, 2, 64, 4, "bf16")
    out, lse = run_selected(case, np.zeros((2, 0), dtype=np.int32), where="k = 0")
    assert (out == 0).all() and torch.isneginf(lse).all()
    out, lse = run_window(case, 4, 0, where="an empty request")
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()
    # more queries than keys: the first queries see nothing
    case = Case(12, [2, 5], 4, 4, 1, 128, 16, "f16")
    out, lse = run_window(case, 0, 0, where="queries before the first key")
    assert (out[:2] == 0).all() and torch.isneginf(lse[:2]).all() and torch.isfinite(lse[2:]).all()


def test_max_seq_len_cuts():
    """Keys at or past max_seq_len are not seen, and a window that lies past it leaves the first tokens."""
    case = Case(13, [300, 40], 2, 8, 2, 128, 16, "f16")
    case.max_seq_len = 64
    run_window(case, 0, 0, where="cut")
    run_window(case, 50, 3, where="cut window")
    run_window(case, 50, 0, where="cut window, nothing left")


def test_bad_pages():
    """Block ids outside the cache hide their keys."""
    case = Case(14, [120, 90], 1, 8, 2, 64, 16, "f16")
    case.table[0, 2], case.table[0, 5], case.table[1, :] = -1, case.n_blocks, 2**31 - 1
    run_window(case, 0, 0, where="bad pages")
    run_selected(case, selection(case, 60), where="bad pages, selected")
    out, lse = run_window(case, 30, 2, where="bad pages, window")
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_nan_stays_with_the_rows_that_see_it(kind):
    """NaN blocks and wild bytes in keys no row may see, and a NaN block that only later rows see."""
    case = Case(15, [70, 37], 4, 8, 2, 128, 16, kind)
    for r in range(2):
        for p in range(int(case.lens[r]), case.table.shape[1] * 16):
            page, off = case.table[r, p // 16], p % 16
            for s in case.scale:
                s[page, off] = 255                       # behind the last key
    free = sorted(set(range(case.n_blocks)) - set(case.table.ravel().tolist()))
    for s in case.scale:
        s[free] = 255                                    # pages no request owns (block 0 too, if it is one)
    run_window(case, 0, 0, where="NaN behind the last key")
    run_window(case, 9, 5, where="NaN behind the last key, window")
    run_selected(case, selection(case, 40), where="NaN behind the last key, selected")
    last = int(case.lens[0]) - 1
    case.scale[1][case.table[0, last // 16], last % 16, 1, 2] = 255     # V, one block: the last query alone sees it
    out, _ = run_window(case, 0, 0, where="V NaN for one row")
    assert torch.isnan(out[3]).any() and not torch.isnan(out[:3]).any()
    case.scale[0][case.table[0, (last - 1) // 16], (last - 1) % 16, 0, 0] = 255  # K: the last two queries
    out, lse = run_window(case, 0, 0, where="K NaN for two rows")
    assert torch.isnan(lse[2:4, :4]).all() and not torch.isnan(lse[:2]).any() and not torch.isnan(lse[4:]).any()
    case.scale[1][case.table[0, 3 // 16], 3, 0, 1] = 255                # V, an early key
    run_window(case, 30, 2, where="V NaN outside the window")
    run_window(case, 0, 0, where="V NaN inside")
    run_selected(case, selection(case, 30), where="V NaN selected or not")


# Sizes at which a wave takes two K/V heads (at most 8 query rows a head, an even
# number of K/V heads, rows * K/V heads >= 1024)
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("query,heads,kv,d,bs", [(1, 32, 16, 64, 16), (1, 128, 16, 128, 7), (2, 16, 16, 96, 32),
                                                 (2, 64, 16, 128, 16)])
def test_pairs_of_heads(query, heads, kv, d, bs, kind):
    rng = np.random.default_rng(d + query)
    lens = [0, 1, 2, 31, 32, 33, 64, 65] + rng.integers(1, 150, 56).tolist()
    case = Case(40, lens, query, heads, kv, d, bs, kind)
    where = f"pairs {query} {heads}/{kv} {d} {kind}"
    run_selected(case, selection(case, 70), where=where)
    run_selected(case, selection(case, 7, 9), 9, where=where + " pooled")
    run_window(case, 0, 0, where=where + " causal")
    run_window(case, 40, 3, where=where + " window")
    # NaN: of one head only, in keys some rows see and others do not
    for which, head, key, block in ((1, 3, 0, 0), (1, 4, 20, d // 32 - 1), (0, 6, 5, 0), (1, 9, 17, 1)):
        for r in (6, 9, 20):
            if key < lens[r]:
                case.scale[which][case.table[r, key // bs], key % bs, head, block] = 255
    out, _ = run_window(case, 40, 3, where=where + " window, NaN")
    assert torch.isnan(out).any()
    run_selected(case, selection(case, 70), where=where + " NaN")


# Sizes at which a wave has the codes of two tiles on the way (129 to 256 pairs of
# a row tile and a K/V head, room for at least 2048 keys), its tiles none to many
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv,d,bs", [(16, 16, 64, 16), (80, 16, 128, 7), (48, 16, 96, 32)])
def test_two_tiles_ahead(heads, kv, d, bs, kind):
    lens = [0, 1, 31, 33, 256, 257, 300, 513, 544, 600, 767, 800, 1025, 40, 900, 1300]
    case = Case(46, lens, 1, heads, kv, d, bs, kind)
    case.max_seq_len = 2100
    more = -(-2100 // bs) - case.table.shape[1]
    case.table = np.concatenate([case.table, np.full((16, more), -1, dtype=np.int32)], 1)
    where = f"two ahead {heads}/{kv} {d} {kind}"
    run_window(case, 0, 0, where=where)
    run_window(case, 2000, 90, where=where + " window")
    run_selected(case, selection(case, 2048), where=where + " selected")
    run_selected(case, selection(case, 256, 9), 9, where=where + " pooled")
    for which, head, key, block in ((1, 3, 0, 0), (1, 4, 20, d // 32 - 1), (0, 6, 5, 0)):
        for r in (7, 9, 15):
            case.scale[which][case.table[r, key // bs], key % bs, head, block] = 255
    out, _ = run_window(case, 0, 0, where=where + " NaN")
    assert torch.isnan(out).any()


# Sizes at which the waves of a workgroup take 2, 4 and 8 K/V heads (more than 16
# query rows a head and request, workgroups that fill the chip)
@pytest.mark.parametrize("requests,kv,kind", [(64, 8, "f16"), (128, 8, "bf16"), (240, 8, "f16"), (120, 2, "bf16")])
def test_groups_of_heads(requests, kv, kind):
    rng = np.random.default_rng(requests)
    lens = rng.integers(1, 90, requests).tolist()
    case = Case(41, lens, 8, 4 * kv, kv, 64, 16, kind)
    args = case.args()
    scale = case.sm_scale
    for window, sinks in ((0, 0), (30, 5)):
        out, lse = li.mx4_attend_window(*args, case.max_seq_len, scale, window=window, sinks=sinks)
        # a request at a time: the same keys in the same tiles of one wave's order or another
        few = [0, 1, requests // 2, requests - 1]
        small = Case(41, [lens[r] for r in few], 8, 4 * kv, kv, 64, 16, kind)
        small.table, small.data, small.scale, small.n_blocks = (case.table[few], case.data, case.scale, case.n_blocks)
        small.max_seq_len = case.max_seq_len
        rows = np.concatenate([np.arange(8 * r, 8 * r + 8) for r in few])
        small.q_t, small.q = case.q_t[torch.from_numpy(rows)], case.q[rows]
        want = small.want(lambda t, v, e: plain.positions_window(v, e, window, sinks))
        pick = torch.from_numpy(rows).to(DEV)
        check((out[pick], lse[pick]), want, kind, 64, f"groups {requests} {kv} {window} {kind}")
        for a in range(0, requests, 7):                     # every row against its own small call
            b = min(requests, a + 7)
            q, kd, ks, vd, vs, table, sl, Q = args
            o, z = li.mx4_attend_window(q[8 * a:8 * b], kd, ks, vd, vs, table[a:b], sl[a:b], Q, case.max_seq_len, scale,
                                        window=window, sinks=sinks)
            # both within the bound of the exact values: at most twice it apart; |V| <= 6 * 2
            assert float((o.float() - out[8 * a:8 * b].float()).abs().max()) <= 2 * (3 * UNIT[kind] + 2.0**-12) * 12
            fine = torch.isfinite(z)
            assert torch.equal(fine, torch.isfinite(lse[8 * a:8 * b]))
            assert float((z - lse[8 * a:8 * b])[fine].abs().max()) <= 2.0**-12


def check_many(case, window, sinks, where, sample, step=1):
    """A call of many rows: `sample` of them against the plain form, and all
    against calls of `step` requests, whose rows another kernel may take."""
    args = case.args()
    q, kd, ks, vd, vs, table, sl, Q = args
    out, lse = li.mx4_attend_window(*args, case.max_seq_len, case.sm_scale, window=window, sinks=sinks)
    few = set(sample.tolist())
    want = case.want(lambda t, v, e: plain.positions_window(v, e, window, sinks) if t in few else [])
    pick = torch.from_numpy(sample).to(DEV)
    o, z, b = want
    b = {k: v[sample] for k, v in b.items()}
    check((out[pick], lse[pick]), (o[sample], z[sample], b), case.kind, case.d, where)
    for a in range(0, len(case.lens), step):
        rows = slice(Q * a, Q * min(a + step, len(case.lens)))
        o, z = li.mx4_attend_window(q[rows], kd, ks, vd, vs, table[a:a + step], sl[a:a + step], Q, case.max_seq_len,
                                    case.sm_scale, window=window, sinks=sinks)
        assert torch.equal(torch.isnan(o), torch.isnan(out[rows])), where
        # each is within 3 roundings of the exact value and 2^-12 for the f32 sums, of at most the largest |V|, 6 * 2
        far = float((o.float() - out[rows].float()).nan_to_num(nan=0.0).abs().max())
        assert far <= 2 * (3 * UNIT[case.kind] + 2.0**-12) * 12, (where, a, far)
        fine = torch.isfinite(z)
        assert torch.equal(fine, torch.isfinite(lse[rows])) and torch.equal(torch.isnan(z), torch.isnan(lse[rows])), where
        assert float((z - lse[rows])[fine].abs().max() if fine.any() else 0.0) <= 2.0**-12, where
    return out, lse


# Sizes at which a workgroup goes through the keys together: 16 requests of 256
# query rows at each of 8 K/V heads
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("query,group,d,bs", [(32, 8, 64, 16), (37, 7, 96, 7), (64, 4, 128, 64), (130, 2, 64, 33)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (70, 3), (64, 200), (200, 64), (4000, 9)])
def test_prompt_rows(query, group, d, bs, window, sinks, kind):
    rng = np.random.default_rng(query)
    lens = [0, 1, query - 1, query, 64, 65, 128, 129] + rng.integers(1, 330, 8).tolist()
    case = Case(42, lens, query, 8 * group, 8, d, bs, kind)
    sample = np.sort(rng.permutation(16 * query)[:40])
    check_many(case, window, sinks, f"prompt {query} {group} {d} {window}+{sinks} {kind}", sample, step=4)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_prompt_rows_share_keys_out(kind):
    """Rows whose keys several workgroups share (a long context, few rows), against the plain form."""
    case = Case(45, [9000], 650, 16, 8, 64, 64, kind)
    check_many(case, 0, 0, f"prompt shares {kind}", np.array([0, 77, 649]))
    check_many(case, 8000, 30, f"prompt shares, window {kind}", np.array([0, 300, 649]))
    # the same rows, 13 to a call, whose keys a wave shares out by itself
    q, kd, ks, vd, vs, table, sl, Q = case.args()
    whole, z = li.mx4_attend_window(q, kd, ks, vd, vs, table, sl, Q, 9000, case.sm_scale)
    for a in (0, 325, 637):
        some = torch.tensor([9000 - 650 + a + 13], dtype=torch.int32, device=DEV)
        o, y = li.mx4_attend_window(q[a:a + 13], kd, ks, vd, vs, table, some, 13, 9000, case.sm_scale)
        assert float((o.float() - whole[a:a + 13].float()).abs().max()) <= 2 * (3 * UNIT[kind] + 2.0**-12) * 12
        assert float((y - z[a:a + 13]).abs().max()) <= 2.0**-12


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_prompt_rows_with_bad_pages_and_nan(kind):
    rng = np.random.default_rng(43)
    lens = [400, 170] + rng.integers(64, 330, 14).tolist()
    case = Case(43, lens, 64, 32, 8, 128, 16, kind)
    sample = np.concatenate([np.arange(0, 128, 9), rng.permutation(896)[:20] + 128])
    case.table[0, 3], case.table[0, 20], case.table[1, 2] = -1, case.n_blocks, 2**30
    check_many(case, 0, 0, "prompt, bad pages", sample, 4)
    check_many(case, 90, 60, "prompt, bad pages, window", sample, 4)
    for r in range(16):                                       # behind the last key
        for p in range(int(case.lens[r]), case.table.shape[1] * 16):
            page = case.table[r, p // 16]
            if 0 <= page < case.n_blocks:
                for s in case.scale:
                    s[page, p % 16] = 255
    out, _ = check_many(case, 0, 0, "prompt, NaN behind the last key", sample, 4)
    assert not torch.isnan(out).any()
    for which, p, head, block in ((1, 390, 0, 3), (1, 100, 1, 0), (0, 370, 1, 2)):
        case.scale[which][case.table[0, p // 16], p % 16, head, block] = 255
    out, lse = check_many(case, 100, 7, "prompt, NaN, window", sample, 4)
    # V at 390: queries 54 on (query j's last key is 336 + j), first K/V head, dimensions 96-127
    assert torch.isnan(out[54:64, :4, 96:]).all() and not torch.isnan(out[:54, :4]).any()
    assert not torch.isnan(out[54:64, :4, :96]).any() and torch.isnan(lse[34:64, 4:8]).all()
    assert not torch.isnan(out[64:]).any() and not torch.isnan(out[:64, 8:]).any()
    check_many(case, 0, 0, "prompt, NaN", sample, 4)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_prompt_rows_of_large_scores(kind):
    rng = np.random.default_rng(44)
    case = Case(44, rng.integers(64, 400, 16).tolist(), 64, 32, 8, 128, 16, kind, spread=40.0)
    sample = np.sort(rng.permutation(1024)[:40])
    for window, sinks in ((0, 0), (150, 5)):
        out, lse = li.mx4_attend_window(*case.args(), case.max_seq_len, case.sm_scale, window=window, sinks=sinks)
        few = set(sample.tolist())
        o, z, b = case.want(lambda t, v, e: plain.positions_window(v, e, window, sinks) if t in few else [])
        pick = torch.from_numpy(sample).to(DEV)
        check((out[pick], lse[pick]), (o[sample], z[sample], {k: v[sample] for k, v in b.items()}), kind, 128,
              f"prompt, large {window} {kind}")
        case.max_seq_len = 250


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_large_scores(kind):
    """Scores in the hundreds: one key takes nearly all the weight, maxima rise through the row."""
    case = Case(16, [600], 2, 8, 2, 128, 16, kind, spread=40.0)
    run_window(case, 0, 0, where="large")
    case = Case(17, [600], 1, 8, 2, 64, 16, kind)
    order = np.argsort((plain.values(case.data[0], case.scale[0])[case.table[0][np.arange(600) // 16],
                                                                  np.arange(600) % 16, 0] @ case.q[0, 0]))
    run_selected(case, order[None].astype(np.int32), where="rising")
    run_selected(case, order[None, ::-1].astype(np.int32).copy(), where="falling")


def test_order_of_the_cache_and_strides():
    """The same attention from a [block][head][slot] cache, padded q and out rows, wider tables."""
    case = Case(18, [130, 77], 2, 8, 4, 96, 16, "bf16")
    q, kd, ks, vd, vs, table, lens, query = case.args()
    want, lse = li.mx4_attend_window(q, kd, ks, vd, vs, table, lens, query, 130, case.sm_scale, window=50, sinks=3)
    turn = lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    wide = torch.zeros((4, 11, 104), dtype=q.dtype, device=DEV)
    wide[:, 2:10, :96] = q
    big = torch.full((4, 8, 112), 3.0, dtype=q.dtype, device=DEV)
    more = torch.cat([table, torch.full((2, 3), -7, dtype=torch.int32, device=DEV)], 1)
    got, _ = li.mx4_attend_window(wide[:, 2:10, :96], turn(kd), turn(ks), turn(vd), turn(vs), more, lens, query, 130,
                                  case.sm_scale, window=50, sinks=3, out=big[:, :, 8:104], with_lse=False)
    assert _ is None and torch.equal(got, want) and torch.equal(big[:, :, 8:104], want)
    assert (big[:, :, :8] == 3.0).all() and (big[:, :, 104:] == 3.0).all()


def test_shared_keys_and_split_rows_agree():
    """One request over many workgroups gives what the plain form gives, and the same bits every time."""
    case = Case(19, [5000], 1, 8, 1, 128, 64, "f16")
    a = run_window(case, 0, 0, where="split")
    for _ in range(3):
        b = run_window(case, 0, 0, where="split")
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    run_window(case, 2000, 7, where="split window")
    run_selected(case, selection(case, 2048), where="split selection")


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv,d", [(3, 1, 64), (20, 2, 96), (5, 1, 192), (40, 2, 256), (17, 1, 256), (4, 4, 128)])
def test_shared_keys_at_every_head_dimension(heads, kv, d, kind):
    """Rows whose keys several workgroups share, each form."""
    case = Case(47, [3300, 2000], 1, heads, kv, d, 32, kind)
    where = f"shares {heads}/{kv} {d} {kind}"
    assert li.mx4_attend_workspace_bytes(2, 1, 3300, False, heads, kv, d) > 0
    run_window(case, 0, 0, where=where)
    run_window(case, 1700, 65, where=where + " window")
    run_selected(case, selection(case, 2000), where=where + " selected")
    run_selected(case, selection(case, 60, 32), 32, where=where + " pooled")
    case.scale[1][case.table[0, 10], 5, kv - 1, d // 32 - 1] = 255
    case.scale[0][case.table[1, 7], 3, 0, 0] = 255
    run_window(case, 0, 0, where=where + " NaN")


def laid_out(case, how):
    """The case's cache in other layouts of the same values."""
    q, kd, ks, vd, vs, table, lens, Q = case.args()
    B, bs, H, w = kd.shape
    sw = ks.shape[3]
    if how == "scales by head":
        ks, vs = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (ks, vs))
    elif how == "scales of a slot together":
        both = torch.stack([ks, vs], 2)
        ks, vs = both[:, :, 0], both[:, :, 1]
    elif how == "one record a slot":
        rec = torch.zeros((B, bs, 2 * H * (w + sw) + 16 - 2 * H * (w + sw) % 16), dtype=torch.uint8, device=DEV)
        step = (bs * rec.shape[2], rec.shape[2])
        parts = [rec.as_strided((B, bs, H, x), step + (x, 1), at)
                 for x, at in ((w, 0), (w, H * w), (sw, 2 * H * w), (sw, 2 * H * w + H * sw))]
        for part, t in zip(parts, (kd, vd, ks, vs)):
            part.copy_(t)
        kd, vd, ks, vs = parts
    elif how == "scales at odd addresses":
        pad = [torch.zeros((B, bs, H, sw + 1), dtype=torch.uint8, device=DEV) for _ in range(2)]
        for p, t in zip(pad, (ks, vs)):
            p[..., 1:] = t
        ks, vs = pad[0][..., 1:], pad[1][..., 1:]
    return q, kd, ks, vd, vs, table, lens, Q


@pytest.mark.parametrize("how", ["scales by head", "scales of a slot together", "one record a slot",
                                 "scales at odd addresses"])
@pytest.mark.parametrize("lens,query,heads,kv,d", [
    ([130, 77], 2, 8, 4, 96),                    # a head at a time
    ([60] * 64, 1, 64, 16, 128),                 # two heads at a time
    ([3000, 900], 1, 16, 2, 128),                # shared keys
    ([200] * 16, 32, 32, 8, 64),                 # many rows
    ([300] * 16, 1, 32, 16, 64),                 # two tiles ahead
])
def test_layouts_of_the_cache(lens, query, heads, kv, d, how):
    case = Case(48, lens, query, heads, kv, d, 16, "bf16")
    if heads == 32 and kv == 16:
        case.max_seq_len = 2048
        case.table = np.concatenate([case.table, np.full((16, 128 - case.table.shape[1]), -1, dtype=np.int32)], 1)
    idx = torch.from_numpy(selection(case, 50)).to(DEV)
    results = []
    for layout in ("as made", how):
        args = laid_out(case, layout)
        results.append(li.mx4_attend_window(*args, case.max_seq_len, case.sm_scale) +
                       li.mx4_attend_window(*args, case.max_seq_len, case.sm_scale, window=40, sinks=3) +
                       li.mx4_attend_selected(*args, idx, case.sm_scale))
    for a, b in zip(*results):
        assert torch.equal(a, b), how


# Sizes at which a workgroup takes a selected row's keys at 8 K/V heads and shares
# their scales (K/V heads a multiple of 8, rows * K/V heads / 8 >= 256 for at most
# 128 keys, 512 or (head dimension 64) 768 for more), tiles of keys none to seven
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("query,heads,kv,d,bs", [(4, 64, 64, 128, 16), (4, 128, 64, 128, 7), (6, 64, 64, 64, 16),
                                                 (12, 128, 32, 64, 33)])
def test_shared_scales(query, heads, kv, d, bs, kind):
    lens = [0, 1, 2, 31, 35, 63, 64, 69, 96, 97, 127, 131, 160, 162, 190, 200]
    case = Case(49, lens, query, heads, kv, d, bs, kind)
    where = f"shared scales {query} {heads}/{kv} {d} {kind}"
    run_selected(case, selection(case, 70), where=where + " few")
    run_selected(case, selection(case, 1), where=where + " one")
    run_selected(case, selection(case, 200), where=where + " many")
    run_selected(case, selection(case, 23, 9), 9, where=where + " pooled")
    run_selected(case, np.full((case.q.shape[0], 40), -1, dtype=np.int32), where=where + " none")
    case.table[12, 1], case.table[14, 2], case.table[15, 0] = -1, case.n_blocks, 2**31 - 1
    # NaN: of one head only, in keys some rows see and others do not
    for which, head, key, block in ((1, 3, 0, 0), (1, 12, 20, d // 32 - 1), (0, 6, 5, 0), (1, 17, 17, 1), (0, 31, 60, 1)):
        for r in (6, 9, 13):
            if key < lens[r]:
                case.scale[which][case.table[r, key // bs], key % bs, head, block] = 255
    out, lse = run_selected(case, selection(case, 200), where=where + " NaN")
    assert torch.isnan(out).any() and torch.isnan(lse).any() and not torch.isnan(out[-query:]).any()
    idx = selection(case, 90)
    first = run_selected(case, idx, where=where + " NaN, few")
    want = case.want(lambda t, v, e: plain.positions_selected(idx[t], 1, e))
    for how in ("scales of a slot together", "one record a slot", "scales by head", "scales at odd addresses"):
        got = li.mx4_attend_selected(*laid_out(case, how), torch.from_numpy(idx).to(DEV), case.sm_scale)
        check(got, want, kind, d, f"{where} {how}")
        if how in ("scales of a slot together", "one record a slot"):    # shared there too
            for a, b in zip(first, got):
                assert torch.equal(a.view(torch.int16), b.view(torch.int16)), how


# Sizes at which they take the same keys under a window (requests * K/V heads / 8
# >= 256, at most 128 keys)
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("query,heads,kv,d,bs", [(1, 128, 64, 128, 16), (2, 64, 64, 96, 7), (3, 128, 64, 64, 33)])
def test_same_keys_under_a_window(query, heads, kv, d, bs, kind):
    lens = [0, 1, 2, 31, 32, 33, 63, 64, 65, 96, 97, 127, 128, 129, 149, 150] * 2
    case = Case(50, lens, query, heads, kv, d, bs, kind)
    where = f"same keys {query} {heads}/{kv} {d} {kind}"
    case.table[12, 1], case.table[31, 0] = -1, 2**31 - 1
    for window, sinks in ((1, 0), (33, 4), (64, 64)):
        run_window(case, window, sinks, where=f"{where} {window}+{sinks}")
    for which, head, key, block in ((1, 3, 0, 0), (1, 12, 20, d // 32 - 1), (0, 6, 5, 0), (1, 47, 30, 1)):
        for r in (6, 9, 13):
            case.scale[which][case.table[r, key // bs], key % bs, head, block] = 255
    out, lse = run_window(case, 100, 10, where=where + " NaN")
    assert torch.isnan(out).any() and torch.isnan(lse).any() and not torch.isnan(out[16 * query:]).any()
    case.max_seq_len = 64                                    # everything, few keys
    run_window(case, 0, 0, where=where + " cut")


def test_a_cache_of_more_than_four_gigabytes():
    """Pages whose bytes lie past 2^32: written, read back and attended to as in a small cache."""
    bs, kv, d = 64, 8, 256
    n_blocks = (2**32 + 2**27) // (bs * kv * d // 2)
    def make(blocks):  # noqa: E306
        return [torch.empty((blocks, bs, kv, w), dtype=torch.uint8, device=DEV) for w in (d // 2, d // 32) * 2]
    big, small = make(n_blocks), make(4)
    assert big[0].numel() > 2**32
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    k, v = (torch.randn((200, kv, d), generator=gen, device=DEV).half() for _ in range(2))
    pages = torch.tensor([n_blocks - 1, 2, n_blocks - 3, n_blocks - 2], device=DEV)
    at = torch.arange(200, device=DEV)
    for cache, table in ((big, pages), (small, torch.arange(4, device=DEV))):
        li.mx4_cache_write(k, table[at // bs] * bs + at % bs, cache[0], cache[1], v, cache[2], cache[3])
    slots = pages[at // bs] * bs + at % bs
    assert torch.equal(li.mx4_cache_read(big[2], big[3], slots), li.mx4_cache_read(small[2], small[3], at))
    q = torch.randn((40, 16, d), generator=gen, device=DEV).half()
    lens = torch.tensor([200], dtype=torch.int32, device=DEV)
    idx = torch.randint(0, 160, (40, 70), generator=gen, device=DEV, dtype=torch.int32)
    results = []
    for cache, table in ((big, pages), (small, torch.arange(4, device=DEV))):
        args = (q, *cache, table.int()[None], lens, 40)
        results.append(li.mx4_attend_window(*args, 200, 0.06) + li.mx4_attend_selected(*args, idx, 0.06))
    for a, b in zip(*results):
        assert torch.equal(a, b)
    # the many-rows form, at a head dimension that has it
    rows = [torch.empty_like(big[0]).view(-1, bs, kv, 64), torch.empty_like(big[1]).view(-1, bs, kv, 4)]
    few = [t[-8:].clone().random_(100, 130) for t in rows]
    for t, f in zip(rows, few):
        t[-8:] = f
    q = torch.randn((2048, 16, 128), generator=gen, device=DEV).half()
    lens = torch.full((16,), 300, dtype=torch.int32, device=DEV)
    own = torch.randint(0, 8, (16, 5), generator=gen, device=DEV)
    got = [li.mx4_attend_window(q, t[0], t[1], t[0], t[1], (own + t[0].shape[0] - 8).int(), lens, 128, 300, 0.09)
           for t in (rows, few)]
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_slots_past_32_bits():
    """A cache of more than 2^31 slots (of one head of 32 values)."""
    n = 2**31 + 4096
    if torch.cuda.mem_get_info()[0] < 60 * 2**30:
        pytest.skip("needs 60 GiB of free GPU memory")
    data = torch.empty((n // 64, 64, 1, 16), dtype=torch.uint8, device=DEV)
    scale = torch.empty((n // 64, 64, 1, 1), dtype=torch.uint8, device=DEV)
    x, v = typed(np.random.default_rng(6).standard_normal((6, 1, 32)), "f16")
    slots = torch.tensor([n - 1, 2**31, 2**31 - 1, 5, n, -1], device=DEV)
    data.view(-1, 16)[-4097:] = 0xA5
    li.mx4_cache_write(x.to(DEV), slots, data, scale)
    got = li.mx4_cache_read(data, scale, slots)
    want = plain.values(*plain.quantise(v, "f16"))
    want[4:] = 0.0
    assert np.array_equal(got.double().cpu().numpy(), want)
    assert (data.view(-1, 16)[-4095:-1] == 0xA5).all()
    del data, scale
    torch.cuda.empty_cache()


def test_largest_windows():
    case = Case(49, [90, 40], 2, 8, 2, 64, 16, "f16")
    whole = run_window(case, 0, 0)
    top = 2**31 - 1
    for window, sinks in ((top, 0), (top, top), (1, top)):
        got = run_window(case, window, sinks, where=f"{window} {sinks}")
        assert torch.equal(got[0], whole[0]) and torch.equal(got[1], whole[1])
    with pytest.raises(ValueError):
        run_window(case, top + 1, 0)


def test_calls_at_once_on_two_streams():
    """Calls with shares of their rows in workspaces, side by side."""
    cases = [Case(50 + i, [4000 + 500 * i], 1, 16, 2, 128, 64, "f16") for i in range(2)]
    args = [c.args() for c in cases]
    want = [li.mx4_attend_window(*a, c.max_seq_len, c.sm_scale) for a, c in zip(args, cases)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(li.mx4_attend_window(*args[i], cases[i].max_seq_len, cases[i].sm_scale))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


def test_pool_and_selection_of_the_whole_row_equal_the_causal_form():
    case = Case(20, [256], 1, 8, 2, 128, 16, "f16")
    whole, _ = run_window(case, 0, 0)
    one, _ = run_selected(case, np.arange(256, dtype=np.int32)[None])
    blocks, _ = run_selected(case, np.arange(8, dtype=np.int32)[None], 32)
    assert torch.equal(one, blocks)                     # the same keys in the same order
    tol = 2 * UNIT["f16"] * (float(whole.abs().max()) + 8)
    assert float((whole.float() - one.float()).abs().max()) <= tol


# ------------------------------------------- used together, streams and graphs

def serve_step(s, out, lse):
    """What a server does for a decode step: write the step's rows, score, select, attend."""
    li.mx4_cache_write(s["k"], s["slots"], s["kd"], s["ks"], s["v"], s["vd"], s["vs"])
    li.score_topk_fused_decode(s["iq"], s["ik"], s["bt"], s["lens"], s["Q"], s["L"], s["w"], s["topk"],
                               workspace=s["ws"], idx=s["idx"], val=s["val"])
    li.mx4_attend_selected(s["q"], s["kd"], s["ks"], s["vd"], s["vs"], s["bt"], s["lens"], s["Q"], s["idx"], s["scale"],
                           out=out[0], lse=lse[0], workspace=s["ws2"])
    li.mx4_attend_window(s["q"], s["kd"], s["ks"], s["vd"], s["vs"], s["bt"], s["lens"], s["Q"], s["L"], s["scale"],
                         window=100, sinks=4, out=out[1], lse=lse[1], workspace=s["ws3"])


def serving(seed, kind="f16"):
    """Requests of a batch whose last keys are written in the step, their index keys already there."""
    import workloads as W
    inp = W.random_decode(seed, 5, 2, 32, 64, 16, 1, 700, 96, w_kind="uniform", max_seq_len=704, poison=False)
    rng = np.random.default_rng(seed)
    H, KV, d, n_blocks, bs = 16, 4, 128, inp.k_cache.shape[0], 16
    on = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    s = dict(iq=on(inp.q), ik=on(inp.k_cache), bt=on(inp.block_table), lens=on(inp.seq_lens), Q=2, L=704, w=on(inp.w),
             topk=96, scale=d**-0.5)
    for n in ("k", "v"):
        s[n + "d"] = on(rng.integers(0, 256, (n_blocks, bs, KV, d // 2), dtype=np.uint8))
        s[n + "s"] = on(rng.integers(123, 129, (n_blocks, bs, KV, d // 32), dtype=np.uint8))
        s[n] = typed(rng.standard_normal((12, KV, d)), kind)[0].to(DEV)
    s["q"] = typed(rng.standard_normal((10, H, d)), kind)[0].to(DEV)
    slots = np.full(12, -1, dtype=np.int64)                                    # a padded batch
    for r in range(5):
        for j in range(2):
            p = int(inp.seq_lens[r]) - 2 + j
            if p >= 0:
                slots[2 * r + j] = int(inp.block_table[r, p // bs]) * bs + p % bs
    s["slots"] = on(slots)
    s["idx"] = torch.full((10, 96), -9, dtype=torch.int32, device=DEV)
    s["val"] = torch.empty((10, 96), device=DEV)
    s["ws"] = torch.empty(li.workspace_bytes(li.OP_FUSED_DECODE, 10, 704, 96), dtype=torch.uint8, device=DEV)
    s["ws2"] = torch.empty(max(256, li.mx4_attend_workspace_bytes(5, 2, 96, True, H, KV, d)), dtype=torch.uint8,
                           device=DEV)
    s["ws3"] = torch.empty(max(256, li.mx4_attend_workspace_bytes(5, 2, 104, False, H, KV, d)), dtype=torch.uint8,
                           device=DEV)
    return s, inp


def results(s):
    rows, H, d = s["q"].shape
    return ([torch.full((rows, H, d), 9.0, dtype=s["q"].dtype, device=DEV) for _ in range(2)],
            [torch.full((rows, H), 9.0, device=DEV) for _ in range(2)])


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_a_decode_step(kind):
    s, inp = serving(21, kind)
    before = s["kd"].clone()
    out, lse = results(s)
    serve_step(s, out, lse)
    torch.cuda.synchronize()
    # the cache: the step's rows as the plain form quantises them, the rest untouched
    slots = s["slots"].cpu().numpy()
    n_blocks, bs, KV, w = s["kd"].shape
    after, old = s["kd"].view(-1, KV, w).cpu().numpy(), before.view(-1, KV, w).cpu().numpy()
    want, _ = plain.quantise(s["k"].double().cpu().numpy(), kind)
    for t, at in enumerate(slots):
        if at >= 0:
            assert np.array_equal(after[at], want[t])
            old[at] = want[t]
    assert np.array_equal(after, old)
    # the attention, from the cache as it now is and the selection as the top-k gave it
    rows = [plain.values(s[n + "d"].cpu().numpy(), s[n + "s"].cpu().numpy()) for n in ("k", "v")]
    idx = s["idx"].cpu().numpy()
    scale = float(np.float32(s["scale"]))
    q = s["q"].double().cpu().numpy()
    for i, positions in enumerate((lambda t, v, e: plain.positions_selected(idx[t], 1, e),
                                   lambda t, v, e: plain.positions_window(v, e, 100, 4))):
        ref = plain.attend_rows(q, *rows, inp.block_table, inp.seq_lens, 2, 704, scale, positions)
        check((out[i], lse[i]), ref, kind, 128, f"step {kind} {i}")


def test_a_decode_step_captured():
    """The step as a graph: replays with new inputs, eager work between, against the eager step."""
    s, _ = serving(22)
    out, lse = results(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        serve_step(s, out, lse)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        serve_step(s, out, lse)
    for step in range(4):
        new, _ = serving(30 + step)
        for name in ("k", "v", "q", "iq"):
            s[name].copy_(new[name])
        for t in out + lse:
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out + lse]
        eager_out, eager_lse = results(s)
        serve_step(s, eager_out, eager_lse)
        torch.cuda.synchronize()
        for a, b in zip(got, eager_out + eager_lse):
            assert torch.equal(a, b), step


def test_on_another_stream():
    case = Case(23, [900, 30], 1, 16, 2, 128, 16, "f16")
    want = run_window(case, 0, 0)
    args = case.args()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = li.mx4_attend_window(*args, case.max_seq_len, case.sm_scale)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ---------------------------------------------------------------- the refusals

def test_binding_refuses():
    case = Case(24, [40, 20], 1, 8, 2, 64, 16, "f16")
    q, kd, ks, vd, vs, bt, sl, Q = case.args()
    idx = torch.zeros((2, 4), dtype=torch.int32, device=DEV)

    def sel(q=q, kd=kd, ks=ks, vd=vd, vs=vs, bt=bt, sl=sl, idx=idx, **kw):
        return li.mx4_attend_selected(q, kd, ks, vd, vs, bt, sl, Q, idx, 0.1, **kw)

    def win(L=40, sl=sl, **kw):
        return li.mx4_attend_window(q, kd, ks, vd, vs, bt, sl, Q, L, 0.1, **kw)

    sel(), win()
    for bad in (dict(q=q.float()), dict(idx=idx.long()), dict(kd=kd.to(torch.int8)), dict(bt=bt.long()),
                dict(sl=sl.long()), dict(q=[1])):
        with pytest.raises(TypeError):
            sel(**bad)
    for bad in (dict(q=q.cpu()), dict(q=q[:1]), dict(idx=idx[:1]), dict(kd=kd[:, :, :1]), dict(ks=ks[:1]),
                dict(vd=vd[:1], vs=vs[:1]), dict(sl=torch.cat([sl, sl])), dict(bt=bt[:1]), dict(kd=kd[0]),
                dict(pool_size=0), dict(out=torch.empty((2, 8, 32), dtype=q.dtype, device=DEV)),
                dict(lse=torch.empty((2, 16), device=DEV)[:, ::2]), dict(idx=idx.repeat(1, 2)[:, ::2]),
                dict(workspace=torch.empty(512, dtype=torch.uint8, device=DEV)[::2])):
        with pytest.raises(ValueError):
            sel(**bad)
    for bad in (dict(L=49 + 16), dict(sl=sl.repeat(2)[::2][:2].flip(0).repeat_interleave(2)[::2])):
        with pytest.raises(ValueError):
            win(**bad)
    for bad in (dict(window=-1), dict(window=4, sinks=-4)):
        with pytest.raises(li.IndexerError):
            win(**bad)
    with pytest.raises(li.IndexerError):
        li.mx4_attend_window(q, kd, ks, vd, vs, bt, sl, Q, 40, float("inf"))
    k = torch.zeros((3, 2, 64), dtype=torch.float16, device=DEV)
    slots = torch.zeros(3, dtype=torch.int64, device=DEV)
    with pytest.raises(TypeError):
        li.mx4_cache_write(k.float(), slots, kd, ks)
    with pytest.raises(TypeError):
        li.mx4_cache_write(k, slots.int(), kd, ks)
    with pytest.raises(TypeError):
        li.mx4_cache_read(kd, ks, slots, torch.float32)
    for call in (lambda: li.mx4_cache_write(k, slots[:2], kd, ks), lambda: li.mx4_cache_write(k, slots, kd, ks, k),
                 lambda: li.mx4_cache_write(k[:, :1], slots, kd, ks),
                 lambda: li.mx4_cache_write(k, slots, kd, ks, k, vd[:1], vs[:1]),
                 lambda: li.mx4_cache_write(k.transpose(1, 2), slots, kd, ks),
                 lambda: li.mx4_cache_read(kd, ks[:1], slots),
                 lambda: li.mx4_cache_read(kd, ks, slots, out=torch.empty((2, 2, 64), dtype=k.dtype, device=DEV)),
                 lambda: li.mx4_cache_read(kd[0], ks, slots)):
        with pytest.raises(ValueError):
            call()


def test_empty_calls():
    case = Case(25, [5], 1, 4, 2, 64, 16, "f16")
    q, kd, ks, vd, vs, bt, sl, Q = case.args()
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    li.mx4_cache_write(torch.empty((0, 2, 64), dtype=q.dtype, device=DEV), none, kd, ks)
    assert li.mx4_cache_read(kd, ks, none).shape == (0, 2, 64)
    slot = torch.zeros(1, dtype=torch.int64, device=DEV)
    assert (li.mx4_cache_read(kd[:0], ks[:0], slot) == 0).all()
    li.mx4_cache_write(torch.ones((1, 2, 64), dtype=q.dtype, device=DEV), slot, kd[:0], ks[:0])
    out, lse = li.mx4_attend_window(q[:0], kd, ks, vd, vs, bt[:0], sl[:0], 1, 5, 0.1)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    out, lse = li.mx4_attend_window(q, kd[:0], ks[:0], vd[:0], vs[:0], bt, sl, 1, 5, 0.1)
    assert (out == 0).all() and torch.isneginf(lse).all()
    out, lse = li.mx4_attend_window(q, kd, ks, vd, vs, bt, sl, 1, 0, 0.1)
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_rows_near_the_limit_of_a_launch():
    """131072 rows of 64 K/V heads of 192: 8.4 million workgroups of 256 threads, half of what a launch holds."""
    rows, H, d, bs = 131072, 64, 192, 16
    if torch.cuda.mem_get_info()[0] < 20 * 2**30:
        pytest.skip("needs 20 GiB of free GPU memory")
    case = Case(51, [40], 1, H, H, d, bs, "f16")
    q, kd, ks, vd, vs, table, lens, _ = case.args()
    idx = torch.full((rows, 2), -1, dtype=torch.int32, device=DEV)
    idx[:, 0] = torch.arange(rows, device=DEV) % 40
    q, table, lens = (t.expand(rows, *t.shape[1:]).contiguous() for t in (q, table, lens))
    out, lse = li.mx4_attend_selected(q, kd, ks, vd, vs, table, lens, 1, idx, case.sm_scale)
    # a row of one key is that key's V
    v = plain.values(case.data[1], case.scale[1])[case.table[0][np.arange(40) // bs], np.arange(40) % bs]
    v = torch.from_numpy(v).to(DEV).half()
    assert torch.isfinite(lse).all()
    for a in range(0, rows, 16384):
        at = torch.arange(a, a + 16384, device=DEV) % 40
        assert torch.equal(out[a:a + 16384], v[at])
    del q, out, lse
    torch.cuda.empty_cache()


def test_more_tokens_than_a_launch_has_workgroups():
    """2^24 + 300 tokens of 5120 values, where one token fills a workgroup of 256 threads: the first and the last
    are written and read back, the others skipped."""
    n, heads, d = 2**24 + 300, 160, 32
    if torch.cuda.mem_get_info()[0] < 10 * 2**30:
        pytest.skip("needs 10 GiB of free GPU memory")
    line = torch.randn(((n + heads) * d,), device=DEV, dtype=torch.float16)
    x = line.as_strided((n, heads, d), (d, d, 1))          # token t's head h is row t + h of one long tensor
    some = torch.cat([torch.arange(5, device=DEV), torch.arange(n - 400, n, 7, device=DEV)])
    slots = torch.full((n,), -1, dtype=torch.int64, device=DEV)
    slots[some] = torch.arange(len(some), device=DEV)
    cache, small = fresh(2, 64, heads, d), fresh(2, 64, heads, d)
    li.mx4_cache_write(x, slots, *cache)
    li.mx4_cache_write(x[some].contiguous(), torch.arange(len(some), device=DEV), *small)
    assert all(torch.equal(a, b) for a, b in zip(cache, small))
    # read: rows without a slot, zeros all, so that they may overlap
    out = torch.full((n + 2 * heads, d), 7.0, device=DEV, dtype=torch.float16)
    slots.fill_(-1)
    got = li.mx4_cache_read(*cache, slots, out=out.as_strided((n, heads, d), (d, d, 1)))
    assert (out[:n + heads - 1] == 0).all() and (out[n + heads - 1:] == 7.0).all() and got.shape == (n, heads, d)
    del line, x, out, got
    torch.cuda.empty_cache()
