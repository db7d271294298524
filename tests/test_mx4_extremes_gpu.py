"""The attention over the 4-bit cache at the ends of its numbers, in every form
of the kernels, against the plain 64-bit forms (bounds: test_mx4_gpu.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import sparse_attention_lightning_indexer_amd as li  # noqa: E402
from oracle import mx4 as plain  # noqa: E402
from mx4_forms import FORMS, agrees, max_keys, meant, taken  # noqa: E402
from test_mx4_gpu import DEV, Case, check, selection  # noqa: E402

SAMPLE = 12   # rows of a large form compared with the plain form; the fewer, the more numbers each reads


def form(name, seed, kind):
    """A case of the form's sizes; its calls take the form, which the test asserts."""
    sizes = FORMS[name]
    for how, want in meant(name).items():
        assert agrees(taken(name, how), want), (name, how)
    case = Case(seed, sizes.lens, sizes.query, sizes.heads, sizes.kv, sizes.d, sizes.bs, kind)
    case.sizes, case.max_seq_len = sizes, sizes.max_seq_len
    more = -(-case.max_seq_len // case.bs) - case.table.shape[1]
    case.table = np.concatenate([case.table, np.full((len(case.lens), more), -1, dtype=np.int32)], 1)
    rows = case.q.shape[0]
    most = int(min(SAMPLE, max(2, 1e7 / (case.heads * max(case.lens) * case.d))))
    case.rows = np.arange(rows) if rows <= 16 else np.sort(case.rng.permutation(rows)[:most])
    if rows > 16:   # the first and last rows of the first request
        case.rows = np.unique(np.concatenate([case.rows, [0, case.query - 1]]))
    return case


def attended(case, how):
    """(the call's out and lse, positions of a row) of a form of the attention."""
    args = case.args()
    if how == "selected":
        idx = selection(case, max_keys(case.sizes, how), holes=0.02)
        got = li.mx4_attend_selected(*args, torch.from_numpy(idx).to(DEV), case.sm_scale)
        return got, lambda t, v, e: plain.positions_selected(idx[t], 1, e)
    window, sinks = (0, 0) if how == "causal" else (case.sizes.window, case.sizes.sinks)
    got = li.mx4_attend_window(*args, case.max_seq_len, case.sm_scale, window=window, sinks=sinks)
    return got, lambda t, v, e: plain.positions_window(v, e, window, sinks)


def numbers(case):
    """K's and V's values."""
    return [plain.values(d, s) for d, s in zip(case.data, case.scale)]


def expected(case, positions, k, v):
    """The plain form of the case's sampled rows."""
    few = set(case.rows.tolist())
    o, z, b = plain.attend_rows(case.q, k, v, case.table, case.lens, case.query, case.max_seq_len, case.sm_scale,
                                lambda t, vis, e: positions(t, vis, e) if t in few else [])
    return o[case.rows], z[case.rows], {n: x[case.rows] for n, x in b.items()}


def sampled(case, got):
    pick = torch.from_numpy(case.rows).to(DEV)
    return tuple(x[pick] for x in got)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("name", list(FORMS))
def test_every_form(name, kind):
    """Ordinary numbers, pages outside the cache, and blocks of NaN that some rows and heads see and others do not."""
    case = form(name, 63, kind)
    kv_values = numbers(case)
    for how in ("causal", "window", "selected"):
        got, positions = attended(case, how)
        check(sampled(case, got), expected(case, positions, *kv_values), kind, case.d, f"{name} {how} {kind}")
    R, kv = len(case.lens), case.kv
    case.table[R // 2, 0] = -1
    case.table[R - 1, (int(case.lens[R - 1]) - 1) // case.bs // 2] = case.n_blocks
    for i, r in enumerate(range(0, R, 2)):
        last = int(case.lens[r]) - 1
        for which, p, head, block in ((1, last, i % kv, 1), (0, last - 1, (i + 1) % kv, 0), (1, 3, (i + 2) % kv, 0)):
            page = case.table[r, p // case.bs]
            if p >= 0 and 0 <= page < case.n_blocks:
                case.scale[which][page, p % case.bs, head, block] = 255
    kv_values = numbers(case)
    for how in ("causal", "window", "selected"):
        got, positions = attended(case, how)
        check(sampled(case, got), expected(case, positions, *kv_values), kind, case.d, f"{name} {how} {kind}, NaN and bad pages")


# V's values end at 6 * 2^13 (f16) and 6 * 2^125 (bf16), scale bytes 140 and 252: the largest
# that the type's own writer stores
ENDS = {"f16": (6 * 2.0**13, (141, 142, 143, 150, 254)), "bf16": (6 * 2.0**125, (253, 254))}


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("name", list(FORMS))
def test_values_past_the_type_stay_with_their_rows(name, kind):
    """V's values that the query's type does not hold (a cache written from another type): rows that do not see
    them, and other heads, are as without them; rows that do take them as the largest value the type's writer
    stores."""
    case = form(name, 60, kind)
    most, scales = ENDS[kind]
    Q, kv, blocks = case.query, case.kv, case.d // 32
    for i, r in enumerate(range(0, len(case.lens), 3)):
        last = int(case.lens[r]) - 1
        # the last key (the last query alone sees it), one out of the window, one among the first
        for p, head, block in ((last, i % kv, i % blocks), (last - case.sizes.window - 7 - Q, (i + 1) % kv, blocks - 1), (4, (i + 2) % kv, 0)):
            if p >= 0:
                case.scale[1][case.table[r, p // case.bs], p % case.bs, head, block] = scales[i % len(scales)]
    hit = False
    k, v = numbers(case)
    v = np.clip(v, -most, most)
    for how in ("causal", "window", "selected"):
        got, positions = attended(case, how)
        out, lse = sampled(case, got)
        o, z, b = expected(case, positions, k, v)
        huge = b["plain"] >= 2.0**100           # bf16: weights times such values pass f32's range in rows that see them
        hit |= bool((b["plain"] >= 40000).any())
        assert torch.isfinite(out[torch.from_numpy(~huge).to(DEV)]).all(), (name, how)
        out = torch.where(torch.from_numpy(huge).to(DEV), torch.from_numpy(o).to(DEV), out.double())
        check((out, lse), (o, z, b), kind, case.d, f"{name} {how} {kind}")
    assert hit


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("name", list(FORMS))
def test_keys_past_the_type_stay_with_their_rows(name, kind):
    """K's values that the query's type does not hold are infinite: rows that do not see them, and other heads, are as
    without them (whatever the rows are that do)."""
    case = form(name, 64, kind)
    _, scales = ENDS[kind]
    kv, blocks = case.kv, case.d // 32
    clean = numbers(case)
    k = clean[0].copy()
    for i, r in enumerate(range(0, len(case.lens), 3)):
        last = int(case.lens[r]) - 1
        for p, head, block in ((last, i % kv, i % blocks), (last - case.sizes.window - 7 - case.query, (i + 1) % kv, blocks - 1),
                               (4, (i + 2) % kv, 0)):
            if p >= 0:
                at = case.table[r, p // case.bs], p % case.bs, head
                case.scale[0][at + (block,)] = scales[i % len(scales)]
                k[at + (slice(32 * block, 32 * block + 32),)] = np.nan
    seen = 0
    for how in ("causal", "window", "selected"):
        got, positions = attended(case, how)
        out, lse = (x.double().cpu() for x in sampled(case, got))
        o, z, b = expected(case, positions, k, clean[1])
        theirs = torch.from_numpy(np.isnan(z))            # rows and heads that attend to such a key
        seen += int(theirs.sum())
        out[theirs], lse[theirs] = float("nan"), float("nan")
        o[np.isnan(z)] = np.nan
        for n in ("reach", "top"):
            b[n] = np.nan_to_num(b[n])
        check((out, lse), (o, z, b), kind, case.d, f"{name} {how} {kind}")
    assert seen


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("name", list(FORMS))
def test_queries_of_nan_and_infinity_stay_alone(name, kind):
    """Rows of a padded batch may hold anything: q of NaN, infinity and the largest number changes its own row and head."""
    case = form(name, 65, kind)
    k, v = numbers(case)
    big = float(torch.finfo(case.q_t.dtype).max)
    theirs = np.zeros(case.q.shape[:2], dtype=bool)
    for i, t in enumerate(case.rows[::2]):
        for h in range(i % 3, case.heads, 5):
            case.q_t[t, h, i % case.d:] = (float("nan"), float("inf"), -float("inf"), big)[(i + h) % 4]
            theirs[t, h] = True
    case.q = np.where(theirs[..., None], 0.0, case.q)
    theirs = theirs[case.rows]
    for how in ("causal", "window", "selected"):
        got, positions = attended(case, how)
        out, lse = (x.double().cpu() for x in sampled(case, got))
        o, z, b = expected(case, positions, k, v)
        out[torch.from_numpy(theirs)], lse[torch.from_numpy(theirs)] = float("nan"), float("nan")
        o[theirs], z[theirs] = np.nan, np.nan
        check((out, lse), (o, z, b), kind, case.d, f"{name} {how} {kind}")


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("name", list(FORMS))
def test_scores_far_from_zero(name, kind):
    """Scores past 2^20: where one key leads by more than the scores' own error, the row is its V, and lse its score."""
    case = form(name, 61, kind)
    k, val = numbers(case)
    for power in (18, 25, 33):
        case.sm_scale = 2.0**power
        assert sum(one_key_rows(case, how, k, val, kind, f"{name} 2^{power}") for how in ("causal", "window", "selected")) > 20


def one_key_rows(case, how, k, val, kind, name):
    """Checks a call; how many of its rows one key decides."""
    checked = 0
    got, positions = attended(case, how)
    out, lse = (x.double().cpu().numpy() for x in sampled(case, got))
    for i, t in enumerate(case.rows):
        r, j = divmod(int(t), case.query)
        vis = int(case.lens[r]) - case.query + 1 + j
        pos = np.array(positions(t, vis, min(vis, case.max_seq_len)), dtype=np.int64)
        if not pos.size:
            continue
        page, off = case.table[r, pos // case.bs], pos % case.bs
        for h in range(0, case.heads, max(1, case.heads // 8)):
            kv = h // (case.heads // case.kv)
            z = case.sm_scale * (k[page, off, kv] @ case.q[t, h])
            reach = case.sm_scale * np.max(np.abs(k[page, off, kv]) @ np.abs(case.q[t, h]))
            error = case.d * 2.0**-23 * reach + 2.0**-22 * np.max(np.abs(z))    # as in test_mx4_gpu.py
            order = np.sort(z)
            lead = order[-1] - order[-2] if z.size > 1 else np.inf
            assert abs(lse[i, h] - order[-1]) <= error + np.log(z.size) + 1, (name, how, t, h, lse[i, h], order[-1])
            if lead <= 2 * error + 120:      # e^-120 of |V| <= 12 is far below half a step of any V but 0
                continue
            want = val[page, off, kv][np.argmax(z)]
            # the weight is rounded to the type, and the result (the weights' sum is not)
            tol = 2 * {"f16": 2.0**-11, "bf16": 2.0**-8}[kind] * np.abs(want) + 2.0**-60
            assert np.all(np.abs(out[i, h] - want) <= tol), (name, how, t, h)
            checked += 1
    return checked


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("name", list(FORMS))
@pytest.mark.parametrize("first", [True, False])
def test_many_small_weights_beside_a_large_one(name, first, kind):
    """One key leads all others by 17.5: each of them weighs 2^-25, less than half of f16's least number, and
    together they are what the row's output is made of.

    f16 weights stand against 2^7 for the largest, so the least number below them is 2^-31 of it, and each is off by
    half of that: 2^-32 sum|V|, with the relative terms and the output's own roundings as in test_mx4_gpu.py."""
    case = form(name, 62, kind)
    case.scale = [np.full_like(s, 127) for s in case.scale]
    case.data[0][:] = 0
    case.data[1][:] = 0x22                       # every value 1
    case.q_t = torch.zeros_like(case.q_t)
    case.q_t[..., 3] = 1.0
    case.q = case.q_t.double().numpy()
    case.sm_scale = float(np.float32(17.5 / 4.0))
    for r, n in enumerate(case.lens):            # the leading key: 4 in dimension 3, V 0
        p = 0 if first else max(0, int(n) - case.query)
        page, off = case.table[r, p // case.bs], p % case.bs
        case.data[0][page, off, :, 1] = 0x60
        case.data[1][page, off] = 0
    kv_values = numbers(case)
    for how in ("causal", "selected"):
        got, positions = attended(case, how)
        o, z, b = expected(case, positions, *kv_values)
        out, lse = (x.double().cpu().numpy() for x in sampled(case, got))
        n = b["count"][:, None]
        unit = {"f16": 2.0**-11, "bf16": 2.0**-8}[kind]
        delta = case.d * 2.0**-23 * b["reach"] + 2.0**-22 * (b["top"] + 1)
        tol = (unit + 2 * delta + (n + 64) * 2.0**-23)[..., None] * b["spread"] + unit * np.abs(o)
        tol = tol + (2.0**-32 * b["plain"] + 2.0**-25 if kind == "f16" else 2.0**-126 * (b["plain"] + 1))
        assert np.all(np.abs(out - o) <= tol), (name, how, float(np.max(np.abs(out - o) / tol)))
        assert (o > 0).any()
        some = np.isfinite(z)
        assert np.array_equal(np.isneginf(lse), ~some)
        assert np.all(np.abs(lse[some] - z[some]) <= (delta + (n + 64) * 2.0**-23 + 2.0**-22 * 20)[some])
