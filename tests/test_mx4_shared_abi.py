"""Attention of requests that share a prefix, on the host: refusals (none of
these calls reaches a launch), workspace sizes, the plain form's own pins."""
import ctypes

import numpy as np
import pytest

import sparse_attention_lightning_indexer_amd as li
from oracle import mx4 as plain
from sparse_attention_lightning_indexer_amd import mx4
from test_mx4_abi import A, B, PAGE_REFUSALS, PAGES, STRIDES, packed


@pytest.fixture(scope="module")
def lib():
    return mx4._library()


def shared(lib, **kw):
    a = dict(q=A, qst=64 * 128, qsh=128, type=0, kd=A, ks=A, vd=B, vs=B, bt=A, bts=8, sl=A, R=2, Q=1, L=128, H=64,
             KV=8, d=128, scale=0.1, idx=None, idxs=0, n=0, pool=0, window=-5, sinks=-5, out=B, ost=64 * 128, osh=128,
             lse=A, ws=A, wsn=1 << 40, stream=None, **PAGES)
    groups = dict(lens=A, starts=A, G=1, most=2, prefix=100)
    a.update({k: v for k, v in kw.items() if k not in groups})
    groups.update({k: v for k, v in kw.items() if k in groups})
    return lib.indexer_mx4_attend_shared(packed(
        mx4.ATTEND, a, "q qst qsh kd ks vd vs " + STRIDES + "bt bts sl out ost osh lse ws wsn stream idx idxs "
        "n pool window sinks type nb bs R Q L H KV d scale") + packed(mx4.SHARED, groups, "lens starts G most prefix"))


# sizes whose rows have shares of the prefix's keys (few keys have none, and no workspace)
LONG = dict(R=64, L=18432, bts=1152, nb=9999, most=64, prefix=16384)


@pytest.mark.parametrize("kw,status,msg", PAGE_REFUSALS + [
    (dict(type=3), li.EINVAL, b"type=3"),
    (dict(R=-1), li.EINVAL, b"n_requests"),
    (dict(KV=7), li.ENOTSUP, b"n_kv_heads=7"),
    (dict(d=160), li.ENOTSUP, b"head_dim=160"),
    (dict(L=2**31 - 1), li.ENOTSUP, b"max_seq_len"),
    (dict(scale=0.0), li.EINVAL, b"sm_scale"),
    (dict(q=None), li.EINVAL, b"q is NULL"),
    (dict(ost=8), li.EINVAL, b"out's row stride"),
    (dict(vs=None), li.EINVAL, b"v_scale is NULL"),
    (dict(bts=7), li.EINVAL, b"bt_stride"),
    (dict(sl=None), li.EINVAL, b"seq_lens is NULL"),
    (dict(G=-1), li.EINVAL, b"n_groups=-1"),
    (dict(most=3), li.EINVAL, b"max_group=3"),
    (dict(most=-1), li.EINVAL, b"max_group=-1"),
    (dict(prefix=-1), li.EINVAL, b"max_prefix_len=-1"),
    (dict(G=2**30), li.EINVAL, b"int32"),
    (dict(lens=None), li.EINVAL, b"prefix_lens is NULL"),
    (dict(starts=None, G=2), li.EINVAL, b"group_starts is NULL"),
    (dict(starts=None, most=1), li.EINVAL, b"max_group=1 is not all"),
    (dict(lens=A + 2), li.EINVAL, b"prefix_lens and group_starts"),
    (dict(starts=A + 1), li.EINVAL, b"prefix_lens and group_starts"),
    (dict(ws=None, **LONG), li.EWORKSPACE, b"workspace"),
    (dict(ws=A + 16, **LONG), li.EWORKSPACE, b"workspace"),
    (dict(wsn=255, **LONG), li.EWORKSPACE, b"workspace"),
])
def test_refuses(lib, kw, status, msg):
    assert shared(lib, **kw) == status
    assert msg in lib.indexer_last_error()


def test_null_arguments_and_no_requests(lib):
    assert lib.indexer_mx4_attend_shared(None) == li.EINVAL
    assert b"args is NULL" in lib.indexer_last_error()
    assert shared(lib, R=0, most=0, ws=None) == li.OK
    assert lib.indexer_last_error() == b""


def test_workspace_bytes(lib):
    f = li.mx4_attend_shared_workspace_bytes
    need = f(64, 1, 18432, 1, 64, 16384, 64, 8, 128)
    assert need % 256 == 0 and need >= 2 * 64 * 64 * 128 * 4            # two shares at least
    assert shared(lib, wsn=need - 1, **LONG) == li.EWORKSPACE
    assert f(2, 1, 128, 1, 2, 100, 64, 8, 128) == 0                     # two requests of few keys: no shares
    assert f(0, 1, 100, 1, 0, 50, 64, 8, 128) == 0
    none = ctypes.c_size_t(-1).value
    for bad in ((-1, 1, 1, 1, 0, 1, 64, 8, 128), (2, 0, 1, 1, 1, 1, 64, 8, 128), (2, 1, -1, 1, 1, 1, 64, 8, 128),
                (2, 1, 1, -1, 1, 1, 64, 8, 128), (2, 1, 1, 1, 3, 1, 64, 8, 128), (2, 1, 1, 1, -1, 1, 64, 8, 128),
                (2, 1, 1, 1, 1, -1, 64, 8, 128), (2, 1, 1, 1, 1, 1, 64, 7, 128), (2, 1, 1, 1, 1, 1, 64, 8, 100),
                (70000, 70000, 1, 1, 1, 1, 64, 8, 128), (2, 1, 1, 2**30, 2, 1, 64, 8, 128)):
        assert f(*bad) == none, bad
    with pytest.raises(ValueError):
        f(2**31, 1, 1, 1, 1, 1, 64, 8, 128)


def test_any_sizes_have_shares_the_join_takes():
    """No plan has more shares of a row than the join adds up, or none of a request's own keys."""
    rng = np.random.default_rng(1)
    f = mx4._library().lidx_mx4_shared_form
    for _ in range(3000):
        requests = int(np.exp(rng.uniform(0, 6)))
        groups = int(rng.integers(1, requests + 1))
        kv, group = int(rng.choice([1, 2, 4, 8, 16])), int(rng.choice([1, 3, 4, 8, 16, 40]))
        prefix = int(np.exp(rng.uniform(0, 13)))
        sizes = (requests, int(rng.choice([1, 2, 4, 64, 500])), prefix + int(np.exp(rng.uniform(0, 13))), groups,
                 int(rng.integers(1, requests + 1)), prefix, kv * group, kv, int(rng.choice([64, 96, 128, 192, 256])))
        out = (ctypes.c_int32 * 16)()
        f((ctypes.c_int32 * 9)(*sizes), out)
        assert out[14] >= 1 and out[6] + out[14] <= 64, sizes


def test_plain_form_by_hand():
    """Two requests of one key of the prefix and one of their own: the second's prefix page is the first's."""
    k = np.zeros((4, 1, 1, 2))
    v = np.arange(8.0).reshape(4, 1, 1, 2)
    table = np.array([[0, 1], [3, 2]], dtype=np.int32)
    q = np.zeros((2, 1, 2))
    out, lse, _ = plain.attend_shared(q, k, v, table, np.array([2, 2]), 1, 2, 1.0, [0, 2], [1])
    assert np.allclose(out[:, 0], [[1.0, 2.0], [2.0, 3.0]]) and np.allclose(lse, np.log(2))
    out, _, _ = plain.attend_shared(q, k, v, table, np.array([2, 2]), 1, 2, 1.0, [0, 1], [1])
    assert np.allclose(out[:, 0], [[1.0, 2.0], [5.0, 6.0]])        # the second is of no group
    out, _, _ = plain.attend_shared(q, k, v, table, np.array([0, 1]), 1, 2, 1.0, [0, 2], [2])
    assert np.allclose(out[:, 0], [[0.0, 0.0], [0.0, 1.0]])
