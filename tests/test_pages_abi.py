"""The page operators on the host: symbols, refusals (none of these calls
reaches a launch), and the plain forms' own pins."""
import ctypes
import os
import re

import numpy as np
import pytest

import sparse_attention_lightning_indexer_amd as li
from oracle import pages as plain
from sparse_attention_lightning_indexer_amd import pages

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "indexer_pages.h")
A, B = 0x10000, 0x20000  # fake, aligned "device" addresses; never dereferenced


@pytest.fixture(scope="module")
def lib():
    return pages._library()


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    assert set(re.findall(r"\b(indexer_[a-z_]+)\s*\(", text)) == set(li.PAGES_EXPORTS)
    assert all(hasattr(lib, n) for n in li.PAGES_EXPORTS)


def arrays(*lists):
    buffer = ctypes.create_string_buffer(b"".join(pages.ARRAY.pack(*a) for a in lists))
    return buffer, ctypes.addressof(buffer)


GOOD = arrays((A, 256, 256), (B, 64, 32))
NO_BASE, NO_BYTES, SHORT, HUGE, FAR = (arrays((A, 256, 256), a) for a in (
    (0, 64, 64), (A, 64, 0), (A, 64, 65), (A, 2**33, 2**31), (A, 2**62, 64)))

CALLS = {
    "copy": (pages.COPY, "arrays from to stream n_arrays n pages"),
    "fork": (pages.FORK, "arrays refs table stride lens parents children fresh stream n_arrays n pages rows cols bs"),
    "grow": (pages.GROW, "refs table stride lens list new slots stream n tokens pages rows cols bs"),
    "free": (pages.FREE, "refs table stride lens list stream n pages rows cols"),
    "compact": (pages.COMPACT, "arrays refs table stride place live ws ws_bytes stream n_arrays pages rows cols"),
}
BASE = dict(arrays=GOOD[1], refs=A, table=A, stride=40, lens=A, parents=A, children=B, fresh=A, list=A, new=0, slots=A,
            place=A, live=B, ws=A, ws_bytes=4 * 101, stream_=0, n_arrays=2, n=3, tokens=5, pages=100, rows=8, cols=40,
            bs=16)
BASE["from"], BASE["to"], BASE["unused"] = A, B, 0


def call(lib, which, **kw):
    layout, names = CALLS[which]
    a = dict(BASE, **kw)
    names = names.split()
    # "stream" is the table's stride's neighbour in name only
    values = [a["stream_"] if n == "stream" else a[n] for n in names]
    return getattr(lib, "indexer_pages_" + which)(layout.pack(*values))


POOL = [(dict(pages=-1), li.EINVAL, b"n_pages"), (dict(pages=2**31 - 1), li.ENOTSUP, b"n_pages")]
ARRAYS = [
    (dict(n_arrays=-1), li.EINVAL, b"n_arrays"),
    (dict(arrays=0), li.EINVAL, b"arrays is NULL"),
    (dict(arrays=NO_BASE[1]), li.EINVAL, b"array 1's base"),
    (dict(arrays=NO_BYTES[1]), li.EINVAL, b"array 1's pages of 0 bytes"),
    (dict(arrays=SHORT[1]), li.EINVAL, b"array 1's stride 64"),
    (dict(arrays=HUGE[1]), li.EINVAL, b"array 1's pages of 2147483648 bytes"),
    (dict(arrays=FAR[1]), li.EINVAL, b"too large"),
]
TABLE = [
    (dict(rows=-1), li.EINVAL, b"n_rows"),
    (dict(cols=-1), li.EINVAL, b"n_cols"),
    (dict(refs=0), li.EINVAL, b"refs is NULL"),
    (dict(refs=A + 2), li.EINVAL, b"refs must be"),
    (dict(table=0), li.EINVAL, b"block_table is NULL"),
    (dict(table=A + 1), li.EINVAL, b"block_table must be"),
    (dict(stride=39), li.EINVAL, b"table_stride"),
    (dict(rows=8193), li.ENOTSUP, b"n_rows=8193"),
]
WIDE = dict(cols=2**29, stride=2**29, bs=1)
LIST = [(dict(n=-1), li.EINVAL, b"n=-1")]
ROWS = LIST + [(dict(n=8193), li.ENOTSUP, b"n=8193"), (dict(lens=0), li.EINVAL, b"seq_lens is NULL"),
               (dict(lens=A + 2), li.EINVAL, b"seq_lens must be")]
BLOCK = [(dict(bs=0), li.EINVAL, b"block_size"), (dict(bs=2**26), li.ENOTSUP, b"n_cols*block_size")]
REFUSALS = {
    "copy": POOL + ARRAYS + LIST + [({"from": 0}, li.EINVAL, b"from is NULL"), (dict(to=B + 2), li.EINVAL, b"to must be")],
    "fork": POOL + ARRAYS + TABLE + ROWS + BLOCK + [
        (dict(parents=0), li.EINVAL, b"parents"), (dict(children=A + 1), li.EINVAL, b"children"),
        (dict(fresh=0), li.EINVAL, b"fresh"), (dict(WIDE, n=9), li.EINVAL, b"9 rows of 536870912 columns")],
    "grow": POOL + TABLE + ROWS + BLOCK + [
        (dict(tokens=-1), li.EINVAL, b"tokens=-1"), (dict(tokens=2**30), li.ENOTSUP, b"n*tokens"),
        (dict(list=0), li.EINVAL, b"rows is NULL"), (dict(slots=A + 4), li.EINVAL, b"slots must be 8-byte"),
        (dict(new=A + 2), li.EINVAL, b"new_tokens")],
    "free": POOL + TABLE + ROWS + [
        (dict(WIDE, n=8), li.EINVAL, b"too large for one launch"), (dict(list=A + 2), li.EINVAL, b"rows must be")],
    "compact": POOL + ARRAYS + TABLE + [
        (dict(place=0), li.EINVAL, b"place"), (dict(live=0), li.EINVAL, b"live"),
        (dict(WIDE, rows=8), li.EINVAL, b"8 rows of 536870912 columns"), (dict(ws=0), li.EWORKSPACE, b"workspace"),
        (dict(ws=A + 2), li.EWORKSPACE, b"workspace"), (dict(ws_bytes=403), li.EWORKSPACE, b"needs 404 bytes")],
}


@pytest.mark.parametrize("which,kw,status,msg", [(w, *r) for w, rs in REFUSALS.items() for r in rs])
def test_refuses(lib, which, kw, status, msg):
    assert call(lib, which, **kw) == status
    assert msg in lib.indexer_last_error()


@pytest.mark.parametrize("which", list(CALLS))
def test_null_arguments(lib, which):
    assert getattr(lib, "indexer_pages_" + which)(None) == li.EINVAL
    assert b"args is NULL" in lib.indexer_last_error()


def test_nothing_to_do_is_a_no_op(lib):
    assert call(lib, "copy", n=0) == li.OK
    assert call(lib, "copy", n_arrays=0, arrays=0) == li.OK
    assert call(lib, "fork", n=0, parents=0, children=0, fresh=0) == li.OK
    assert call(lib, "grow", n=0, list=0) == li.OK
    assert call(lib, "grow", tokens=0) == li.OK
    assert call(lib, "free", n=0, list=0) == li.OK
    assert lib.indexer_last_error() == b""


def test_workspace_bytes(lib):
    assert [li.pages_compact_workspace_bytes(n) for n in (0, 1, 2, 5, 100)] == [4, 4, 12, 20, 404]
    assert lib.indexer_pages_compact_workspace_bytes(-1) == ctypes.c_size_t(-1).value
    with pytest.raises(ValueError):
        li.pages_compact_workspace_bytes(2**31)


def test_plain_forms_by_hand():
    """A prompt of 5 tokens in pages of 2, forked twice, grown, freed, compacted."""
    caches = [np.arange(8)[:, None] * 10]
    refs, table, lens = [0, 0, 1, 0, 1, 1, 0, 0], [[4, 2, 5, -1], [-1] * 4, [-1] * 4], [5, 0, 0]
    assert plain.fork(caches, refs, table, lens, [0, 0, 0, 9], [1, 2, 1, 1], 2) == [0, 1, -3, -3]
    assert table == [[4, 2, 5, -1], [4, 2, 0, -1], [4, 2, 1, -1]] and lens == [5, 5, 5]
    assert refs == [1, 1, 3, 0, 3, 1, 0, 0] and caches[0][:, 0].tolist() == [50, 50, 20, 30, 40, 50, 60, 70]
    assert plain.grow(refs, table, lens, [2, 1], 2, 2, [2, 1]) == [[3, 6], [1, -1]]
    assert table[2] == [4, 2, 1, 3] and lens == [5, 6, 7] and refs == [1, 1, 3, 1, 3, 1, 0, 0]
    plain.free(refs, table, lens, [0, 0, -1, 3])
    assert refs == [1, 1, 2, 1, 2, 0, 0, 0] and table[0] == [-1] * 4 and lens == [0, 6, 7]
    plain.free(refs, table, lens, [1])
    assert refs == [0, 1, 1, 1, 1, 0, 0, 0]
    assert plain.compact(caches, refs, table) == ([-1, 1, 2, 3, 0, -1, -1, -1], 4)
    assert table[2] == [0, 2, 1, 3] and refs == [1, 1, 1, 1, 0, 0, 0, 0] and caches[0][0, 0] == 40


def test_plain_forms_out_of_pages():
    refs, table, lens = [1, 0], [[0, -1], [-1, -1], [-1, -1]], [1, 0, 0]
    caches = [np.zeros((2, 1))]
    assert plain.fork(caches, refs, table, lens, [0, 0], [1, 2], 2) == [1, -2]
    assert table[2] == [-1, -1] and lens == [1, 1, 0] and refs == [1, 1]
    # the second row has no page; the third needs none; a full row has no column
    assert plain.grow(refs, table, lens, [1, 2, 0], 1, 2) == [[3], [-1], [1]] and lens == [2, 2, 0]
    refs[1] = 0
    assert plain.grow(refs, table, [4, 0, 0], [0], 1, 2) == [[-1]]
