"""The head norm and rotation on the host: symbols, refusals (none of these
calls reaches a launch), and the plain form's own pins."""
import os
import re

import numpy as np
import pytest

import sparse_attention_lightning_indexer_amd as li
from oracle import rope as plain
from sparse_attention_lightning_indexer_amd import rope

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "indexer_rope.h")
A, B = 0x10000, 0x20000  # fake, aligned "device" addresses; never dereferenced


@pytest.fixture(scope="module")
def lib():
    return rope._library()


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    assert set(re.findall(r"\b(indexer_[a-z_]+)\s*\(", text)) == set(li.ROPE_EXPORTS)
    assert all(hasattr(lib, n) for n in li.ROPE_EXPORTS)


MEMBERS = ("q qst qsh k kst ksh qo qost qosh ko kost kosh qw kw pos ps inv a0 a1 a2 a3 stream type n hq hk d m axes "
           "inter p64 qwt kwt eps scale").split()


def call(lib, **kw):
    a = dict(q=A, qst=1024, qsh=128, k=A, kst=256, ksh=128, qo=B, qost=1024, qosh=128, ko=B, kost=256, kosh=128, qw=A,
             kw=A, pos=A, ps=0, inv=A, a0=0, a1=0, a2=0, a3=0, stream=0, type=0, n=3, hq=8, hk=2, d=128, m=64, axes=1,
             inter=0, p64=1, qwt=0, kwt=0, eps=1e-6, scale=1.0)
    a.update(kw)
    return lib.indexer_norm_rope(rope.NORM_ROPE.pack(*(a[name] for name in MEMBERS)))


@pytest.mark.parametrize("kw,status,msg", [
    (dict(type=2), li.EINVAL, b"type=2"),
    (dict(n=-1), li.EINVAL, b"n_tokens"),
    (dict(hq=0), li.ENOTSUP, b"n_q_heads=0"),
    (dict(hk=1025), li.ENOTSUP, b"n_k_heads=1025"),
    (dict(d=4), li.ENOTSUP, b"head_dim=4"),
    (dict(d=100), li.ENOTSUP, b"head_dim=100"),
    (dict(d=264), li.ENOTSUP, b"head_dim=264"),
    (dict(m=6), li.ENOTSUP, b"n_freq=6"),
    (dict(m=68), li.ENOTSUP, b"n_freq=68"),
    (dict(m=-4), li.ENOTSUP, b"n_freq=-4"),
    (dict(axes=0), li.ENOTSUP, b"n_axes=0"),
    (dict(axes=5), li.ENOTSUP, b"n_axes=5"),
    (dict(axes=2, ps=2), li.EINVAL, b"pos_stride"),
    (dict(axes=2, ps=3, a1=2 << 62), li.EINVAL, b"axis 2 of frequency 63"),
    (dict(a0=1), li.EINVAL, b"axis 1 of frequency 0"),
    (dict(eps=-1.0), li.EINVAL, b"eps"),
    (dict(eps=float("nan")), li.EINVAL, b"eps"),
    (dict(scale=float("inf")), li.EINVAL, b"rotary_scale"),
    (dict(q=0), li.EINVAL, b"q is NULL"),
    (dict(q=A + 8), li.EINVAL, b"q must be 16-byte"),
    (dict(qsh=120), li.EINVAL, b"q's head stride"),
    (dict(qst=0), li.EINVAL, b"q's row stride"),
    (dict(qo=0), li.EINVAL, b"q_out is NULL"),
    (dict(qosh=132), li.EINVAL, b"q_out's head stride"),
    (dict(kst=100), li.EINVAL, b"k's row stride"),
    (dict(ko=0), li.EINVAL, b"k_out is NULL"),
    (dict(kost=-256), li.EINVAL, b"k_out's row stride"),
    (dict(qw=A + 2), li.EINVAL, b"q_weight"),
    (dict(kw=A + 1, kwt=1), li.EINVAL, b"k_weight"),
    (dict(kwt=2), li.EINVAL, b"k_weight's type 2"),
    (dict(pos=0), li.EINVAL, b"positions is NULL"),
    (dict(pos=A + 4), li.EINVAL, b"positions must be aligned"),
    (dict(p64=2), li.EINVAL, b"positions_64"),
    (dict(inv=0), li.EINVAL, b"inv_freq"),
    (dict(n=2**26 + 5, hk=2), li.EINVAL, b"too large"),
])
def test_refuses(lib, kw, status, msg):
    assert call(lib, **kw) == status
    assert msg in lib.indexer_last_error()


@pytest.mark.parametrize("heads,d,m", [(1, 8, 4), (2, 128, 64), (72, 128, 64), (2048, 256, 128), (32, 80, 40)])
def test_the_most_tokens(lib, heads, d, m):
    """2^26 - 4 tokens fit a launch of fewer than 2^32 threads, whatever a row is; the next ones are refused."""
    fits = [lib.lidx_rope_fits(n, heads, d, m) for n in (1, 2**20, 2**26 - 5, 2**26 - 4, 2**26 - 3, 2**26, 2**31 - 1)]
    assert fits == [1, 1, 1, 1, 0, 0, 0]
    q, k = (heads, 0) if heads == 1 else (heads // 2, heads - heads // 2)
    for n in (2**26 - 3, 2**26 - 1, 2**31 - 1):
        assert call(lib, n=n, hq=q, hk=k, k=A if k else 0, d=d, m=m, qsh=256, ksh=256, qosh=256, kosh=256, qst=2**19,
                    kst=2**19, qost=2**19, kost=2**19) == li.EINVAL
        assert b"too large" in lib.indexer_last_error()


def test_null_arguments(lib):
    assert lib.indexer_norm_rope(None) == li.EINVAL
    assert b"args is NULL" in lib.indexer_last_error()


def test_nothing_to_do_is_a_no_op(lib):
    assert call(lib, n=0) == li.OK
    assert call(lib, n=0, k=0, ko=0, hk=0, m=0, pos=0, inv=0) == li.OK
    assert lib.indexer_last_error() == b""


def test_axis_words():
    axes = tuple(i % 4 for i in range(128))
    words = rope._axis_words(axes)
    assert [(words[i >> 5] >> (2 * (i & 31))) & 3 for i in range(128)] == list(axes)
    for bad in ((4,), (-1,), (0,) * 129, (1.0,)):
        with pytest.raises(ValueError):
            rope._axis_words(bad)


def test_plain_form_by_hand():
    # a quarter turn of (3, 4) with neighbours and halves, the rest passes
    x = np.array([[[3.0, 4.0, 5.0, 6.0]]])
    quarter = np.array([np.pi / 2])
    out, _, _ = plain.norm_rope(x, None, np.array([[1]]), quarter, [0], 0.0, True, 1.0)
    assert np.allclose(out[0, 0], [-4.0, 3.0, 5.0, 6.0])
    out, _, _ = plain.norm_rope(x, None, np.array([[-1]]), quarter, [0], 0.0, False, 2.0)
    assert np.allclose(out[0, 0], [8.0, -6.0, 5.0, 6.0])
    # two axes, and the norm: mean square of (3, 4, 5, 6) is 21.5
    out, _, _ = plain.norm_rope(x, np.array([1.0, 2.0, 1.0, 1.0]), np.array([[0], [2]]), np.array([1.0, np.pi / 2]),
                                [0, 1], 0.0, False, 1.0)
    assert np.allclose(out[0, 0] * np.sqrt(21.5), [3.0, -8.0, 5.0, -6.0])
