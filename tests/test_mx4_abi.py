"""The 4-bit cache operators on the host: symbols, refusals (none of these
calls reaches a launch), workspace sizes, and the plain forms' own pins."""
import ctypes
import os
import re

import numpy as np
import pytest

import sparse_attention_lightning_indexer_amd as li
from oracle import mx4 as plain
from sparse_attention_lightning_indexer_amd import mx4

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "indexer_mx4.h")

A, B = 0x10000, 0x20000  # fake, aligned "device" addresses; never dereferenced


@pytest.fixture(scope="module")
def lib():
    return mx4._library()


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(indexer_mx4_[a-z_]+)\s*\(", text))
    assert names == set(li.MX4_EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


PAGES = dict(nb=4, bs=16, dsb=16 * 8 * 64, dss=8 * 64, dsh=64, ssb=16 * 8 * 4, sss=8 * 4, ssh=4)


def packed(layout, a, names):
    """The argument structure of the members `names` of `a`, in the header's order."""
    return layout.pack(*(0 if a[n] is None else a[n] for n in names.split()))


STRIDES = "dsb dss dsh ssb sss ssh "


def write(lib, **kw):
    a = dict(k=A, kst=1024, ksh=128, v=B, vst=1024, vsh=128, type=0, n=2, H=8, d=128, slots=A, kd=A, ks=A, vd=B, vs=B,
             stream=None, **PAGES)
    a.update(kw)
    return lib.indexer_mx4_cache_write(packed(
        mx4.WRITE, a, "k kst ksh v vst vsh slots kd ks vd vs " + STRIDES + "stream type n H d nb bs"))


PAGE_REFUSALS = [
    (dict(nb=-1), li.EINVAL, b"n_blocks"),
    (dict(bs=0), li.EINVAL, b"block_size"),
    (dict(dsh=72), li.EINVAL, b"multiples of 16"),
    (dict(dsh=48), li.EINVAL, b"data strides"),
    (dict(dss=0), li.EINVAL, b"data strides"),
    (dict(dsb=-1024), li.EINVAL, b"data strides"),
    (dict(ssh=3), li.EINVAL, b"scale strides"),
    (dict(sss=0), li.EINVAL, b"scale strides"),
    (dict(bs=1 << 24), li.ENOTSUP, b"pages not supported"),
    (dict(dss=1 << 24), li.ENOTSUP, b"pages not supported"),
    (dict(sss=1 << 24), li.ENOTSUP, b"pages not supported"),
    (dict(dsh=1 << 30), li.ENOTSUP, b"pages not supported"),
    (dict(dsb=1 << 32), li.ENOTSUP, b"pages not supported"),
    (dict(ssb=1 << 32), li.ENOTSUP, b"pages not supported"),
]


@pytest.mark.parametrize("kw,status,msg", PAGE_REFUSALS + [
    (dict(type=2), li.EINVAL, b"type=2"),
    (dict(n=-1), li.EINVAL, b"n_tokens"),
    (dict(H=0), li.ENOTSUP, b"n_heads=0"),
    (dict(H=1025), li.ENOTSUP, b"n_heads=1025"),
    (dict(d=16), li.ENOTSUP, b"head_dim=16"),
    (dict(d=100), li.ENOTSUP, b"head_dim=100"),
    (dict(d=1056), li.ENOTSUP, b"head_dim=1056"),
    (dict(k=None), li.EINVAL, b"k is NULL"),
    (dict(k=A + 8), li.EINVAL, b"16-byte"),
    (dict(ksh=120), li.EINVAL, b"head stride"),
    (dict(ksh=132), li.EINVAL, b"head stride"),
    (dict(kst=0), li.EINVAL, b"row stride"),
    (dict(vst=1001), li.EINVAL, b"v's row stride"),
    (dict(slots=None), li.EINVAL, b"slots is NULL"),
    (dict(slots=A + 4), li.EINVAL, b"8-byte"),
    (dict(kd=None), li.EINVAL, b"k_data is NULL"),
    (dict(ks=None), li.EINVAL, b"k_scale is NULL"),
    (dict(vd=B + 8), li.EINVAL, b"v_data must be"),
    (dict(vs=None), li.EINVAL, b"v_scale is NULL"),
])
def test_write_refuses(lib, kw, status, msg):
    assert write(lib, **kw) == status
    assert msg in lib.indexer_last_error()


def test_nothing_to_write_is_a_no_op(lib):
    assert write(lib, n=0) == li.OK
    assert write(lib, nb=0, kd=None, ks=None, vd=None, vs=None) == li.OK
    assert lib.indexer_last_error() == b""


def read(lib, **kw):
    a = dict(data=A, scale=A, slots=A, n=2, H=8, d=128, out=B, ost=1024, osh=128, type=1, stream=None, **PAGES)
    a.update(kw)
    return lib.indexer_mx4_cache_read(packed(
        mx4.READ, a, "data scale " + STRIDES + "slots out ost osh stream type n H d nb bs"))


@pytest.mark.parametrize("kw,status,msg", PAGE_REFUSALS + [
    (dict(type=-1), li.EINVAL, b"type=-1"),
    (dict(n=-2), li.EINVAL, b"n_rows"),
    (dict(nb=0), li.EINVAL, b"n_blocks"),
    (dict(d=48), li.ENOTSUP, b"head_dim=48"),
    (dict(out=None), li.EINVAL, b"out is NULL"),
    (dict(out=B + 2), li.EINVAL, b"out must be 16-byte"),
    (dict(osh=124), li.EINVAL, b"out's head stride"),
    (dict(data=None), li.EINVAL, b"data is NULL"),
    (dict(scale=None), li.EINVAL, b"scale is NULL"),
    (dict(slots=None), li.EINVAL, b"slots is NULL"),
])
def test_read_refuses(lib, kw, status, msg):
    assert read(lib, **kw) == status
    assert msg in lib.indexer_last_error()


def test_nothing_to_read_is_a_no_op(lib):
    assert read(lib, n=0) == li.OK


def attend(lib, form, **kw):
    a = dict(q=A, qst=64 * 128, qsh=128, type=0, kd=A, ks=A, vd=B, vs=B, bt=A, bts=8, sl=A, R=2, Q=1, L=128, H=64,
             KV=8, d=128, scale=0.1, idx=A, idxs=32, n=32, pool=1, window=0, sinks=0, out=B, ost=64 * 128, osh=128,
             lse=A, ws=A, wsn=1 << 40, stream=None, **PAGES)
    a.update(kw)
    entry = lib.indexer_mx4_attend_selected if form == "selected" else lib.indexer_mx4_attend_window
    return entry(packed(
        mx4.ATTEND, a, "q qst qsh kd ks vd vs " + STRIDES + "bt bts sl out ost osh lse ws wsn stream idx idxs "
        "n pool window sinks type nb bs R Q L H KV d scale"))


@pytest.mark.parametrize("form", ["selected", "window"])
@pytest.mark.parametrize("kw,status,msg", PAGE_REFUSALS + [
    (dict(type=3), li.EINVAL, b"type=3"),
    (dict(R=-1), li.EINVAL, b"n_requests"),
    (dict(Q=0), li.EINVAL, b"query_len"),
    (dict(L=-1), li.EINVAL, b"max_seq_len"),
    (dict(L=2**31 - 1), li.ENOTSUP, b"max_seq_len"),
    (dict(H=0), li.ENOTSUP, b"n_heads=0"),
    (dict(H=1032), li.ENOTSUP, b"n_heads=1032"),
    (dict(KV=0), li.ENOTSUP, b"n_kv_heads=0"),
    (dict(KV=7), li.ENOTSUP, b"n_kv_heads=7"),
    (dict(d=32), li.ENOTSUP, b"head_dim=32"),
    (dict(d=160), li.ENOTSUP, b"head_dim=160"),
    (dict(R=70000, Q=70000), li.EINVAL, b"int32"),
    (dict(scale=0.0), li.EINVAL, b"sm_scale"),
    (dict(scale=-1.0), li.EINVAL, b"sm_scale"),
    (dict(scale=float("nan")), li.EINVAL, b"sm_scale"),
    (dict(scale=3e38), li.EINVAL, b"sm_scale"),
    (dict(q=None), li.EINVAL, b"q is NULL"),
    (dict(q=A + 8), li.EINVAL, b"q must be 16-byte"),
    (dict(qsh=100), li.EINVAL, b"q's head stride"),
    (dict(out=None), li.EINVAL, b"out is NULL"),
    (dict(ost=8), li.EINVAL, b"out's row stride"),
    (dict(kd=None), li.EINVAL, b"k_data is NULL"),
    (dict(vs=None), li.EINVAL, b"v_scale is NULL"),
    (dict(bt=None), li.EINVAL, b"block_table is NULL"),
    (dict(bts=7), li.EINVAL, b"bt_stride"),
    (dict(sl=None), li.EINVAL, b"seq_lens is NULL"),
    (dict(sl=A + 2), li.EINVAL, b"4-byte"),
    (dict(lse=A + 1), li.EINVAL, b"lse must be"),
])
def test_attend_refuses(lib, form, kw, status, msg):
    assert attend(lib, form, **kw) == status
    assert msg in lib.indexer_last_error()


@pytest.mark.parametrize("kw,status,msg", [
    (dict(n=-1), li.EINVAL, b"n_sel"),
    (dict(pool=0), li.EINVAL, b"pool_size=0"),
    (dict(pool=8193), li.ENOTSUP, b"pool_size=8193"),
    (dict(n=2**20, idxs=2**20, pool=8192), li.ENOTSUP, b"n_sel*pool_size"),
    (dict(idx=None), li.EINVAL, b"idx is NULL"),
    (dict(idx=A + 2), li.EINVAL, b"idx must be"),
    (dict(idxs=31), li.EINVAL, b"idx_stride"),
])
def test_attend_selected_refuses(lib, kw, status, msg):
    assert attend(lib, "selected", **kw) == status
    assert msg in lib.indexer_last_error()


@pytest.mark.parametrize("kw", [dict(window=-1), dict(sinks=-1)])
def test_attend_window_refuses(lib, kw):
    assert attend(lib, "window", **kw) == li.EINVAL
    assert b"window" in lib.indexer_last_error()


def test_attend_refuses_what_one_launch_cannot_hold(lib):
    many = dict(R=2_000_000, H=64, KV=16, ost=64 * 128, idxs=32, n=32)     # 2 million rows of 16 K/V heads
    many.update(dsb=16 * 16 * 64, dss=16 * 64, ssb=16 * 16 * 4, sss=16 * 4, KV=16, H=160, qst=160 * 128, ost=160 * 128)
    assert attend(lib, "selected", **many) == li.EINVAL
    assert b"too large for one launch" in lib.indexer_last_error()


def test_attend_needs_its_workspace(lib):
    need = li.mx4_attend_workspace_bytes(1, 1, 131072, False, 64, 8, 128)
    assert need > 0 and need % 256 == 0
    big = dict(R=1, L=131072, bts=8192, nb=8192)
    for kw in (dict(ws=None), dict(wsn=need - 1), dict(ws=A + 16)):
        assert attend(lib, "window", **big, **kw) == li.EWORKSPACE
        assert b"workspace" in lib.indexer_last_error()
    need = li.mx4_attend_workspace_bytes(2, 1, 2048, True, 64, 8, 128)
    assert need > 0
    assert attend(lib, "selected", n=2048, idxs=2048, wsn=need - 1) == li.EWORKSPACE


def test_no_arguments(lib):
    for name in li.MX4_EXPORTS[:4]:
        assert getattr(lib, name)(None) == li.EINVAL
        assert b"args is NULL" in lib.indexer_last_error()


def test_binding_refuses_what_a_member_cannot_hold():
    for layout, members in ((mx4.READ, [0] * 18 + [2**31]), (mx4.ATTEND, [0] * 38 + [1e39]),
                            (mx4.WRITE, [2**63] + [0] * 23)):
        with pytest.raises(ValueError, match="out of its range"):
            mx4._pack(layout, *members)


def test_no_requests_is_a_no_op(lib):
    for form in ("selected", "window"):
        assert attend(lib, form, R=0, ws=None, wsn=0) == li.OK
    assert lib.indexer_last_error() == b""


def test_workspace_bytes():
    none = ctypes.c_size_t(-1).value
    f = mx4._library().indexer_mx4_attend_workspace_bytes
    assert f(1, 1, 32, 1, 64, 8, 128) == 0             # one tile: nothing to share out
    assert f(4096, 1, 2048, 1, 64, 8, 128) == 0        # rows enough
    assert f(0, 1, 2048, 1, 64, 8, 128) == 0
    for bad in ((-1, 1, 1, 1, 64, 8, 128), (1, 0, 1, 1, 64, 8, 128), (1, 1, -1, 1, 64, 8, 128),
                (1, 1, 1, 1, 64, 7, 128), (1, 1, 1, 1, 64, 8, 100), (1, 1, 1, 1, 0, 1, 128),
                (70000, 70000, 1, 1, 64, 8, 128)):
        assert f(*bad) == none, bad


# ------------------------------------------------- pins of the plain forms

def test_codes_by_hand():
    # middles go to the even code: .25 -> 0, .75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    for y, want in ((0.0, 0), (0.25, 0), (0.2500001, 1), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6),
                    (5.0000001, 7), (6.0, 7), (6.999, 7), (100.0, 7), (-0.0, 8), (-0.75, 10), (-9.0, 15)):
        assert plain.code(y) == want, y
    for i, m in enumerate(plain.MAGNITUDES):
        assert plain.code(float(m)) == i


def test_exponents_by_hand():
    assert plain.exponent(6.99, "f16") == 0 and plain.exponent(7.0, "f16") == 1
    assert plain.exponent(3.5, "bf16") == 0 and plain.exponent(3.49, "bf16") == -1
    assert plain.exponent(0.0, "f16") == -23 and plain.exponent(0.0, "bf16") == -126
    assert plain.exponent(65504.0, "f16") == 13 and plain.exponent(3.3e38, "bf16") == 125


def test_quantise_by_hand():
    x = np.zeros((2, 32), dtype=np.float16)
    x[0, :4] = [7.0, -3.0, 1.5, 0.5]        # scale 2: 3.5 -> 4, -1.5, .75 -> 1, .25 -> 0
    x[1, 5] = np.nan
    data, scale = plain.quantise(x, "f16")
    assert scale.tolist() == [[128], [255]]
    assert data[0, 0] == 6 | ((8 + 3) << 4) and data[0, 1] == 2 | (0 << 4) and not data[0, 2:].any()
    v = plain.values(data, scale)
    assert v[0, :4].tolist() == [8.0, -3.0, 2.0, 0.0] and np.isnan(v[1]).all()


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_no_value_is_off_by_more_than_half_a_step(kind):
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((64, 32)) * np.exp2(rng.integers(-12, 12, (64, 1)))).astype(np.float16)
    data, scale = plain.quantise(x, kind)
    v, unit = plain.values(data, scale), np.ldexp(1.0, scale.astype(int) - 127)
    a = np.abs(x.astype(np.float64)) / unit
    step = np.where(a <= 2, 0.5, np.where(a <= 4, 1.0, 2.0))
    assert np.all(np.abs(v - x) <= 0.5 * step * unit)
    assert np.array_equal(v, v.astype(np.float16))                    # every stored value is of the type
    again = plain.quantise(v, kind)
    assert np.array_equal(plain.values(*again), v)                    # and stays what it is


def test_attention_of_equal_scores_is_the_mean():
    rng = np.random.default_rng(1)
    v = rng.standard_normal((3, 4, 1, 64))
    q, k = np.zeros((2, 2, 64)), rng.standard_normal((3, 4, 1, 64))
    bt = np.array([[2, 0, 1]])
    out, lse, _ = plain.attend_rows(q, k, v, bt, [9], 2, 12, 0.5, lambda t, s, e: plain.positions_window(s, e, 0, 0))
    flat = v[bt[0]].reshape(12, 64)
    np.testing.assert_allclose(out[0], np.broadcast_to(flat[:8].mean(0), (2, 64)), rtol=1e-12)
    np.testing.assert_allclose(out[1], np.broadcast_to(flat[:9].mean(0), (2, 64)), rtol=1e-12)
    np.testing.assert_allclose(lse, np.log([[8, 8], [9, 9]]), rtol=1e-12)


def test_positions_by_hand():
    assert plain.positions_selected([3, -1, 0, 9], 1, 5) == [3, 0]
    assert plain.positions_selected([1, 0], 4, 6) == [4, 5, 0, 1, 2, 3]
    assert plain.positions_window(6, 6, 2, 1) == [0, 4, 5]
    assert plain.positions_window(9, 6, 2, 1) == [0]           # the window lies past the last key kept
    assert plain.positions_window(6, 6, 0, 3) == list(range(6))
    assert plain.positions_window(-1, -1, 4, 4) == []


# ------------------------------------------------- sizes at the ends of their ranges

@pytest.mark.parametrize("kw", [dict(dsh=1 << 62), dict(ssh=1 << 62), dict(dsh=1 << 62, ssh=1 << 62),
                                dict(dsh=(1 << 62) + (1 << 33)), dict(dss=1 << 60, bs=17), dict(sss=1 << 60, bs=17)])
def test_strides_whose_extent_passes_64_bits(lib, kw):
    """5 heads 2^62 bytes apart: their extent is 2^64, which 64 bits hold as 0."""
    for call in (lambda: write(lib, H=5, kst=640, vst=640, **kw), lambda: read(lib, H=5, ost=640, **kw),
                 lambda: attend(lib, "selected", H=5, KV=5, qst=640, ost=640, **kw),
                 lambda: attend(lib, "window", H=5, KV=5, qst=640, ost=640, **kw)):
        assert call() == li.ENOTSUP
        assert b"pages not supported" in lib.indexer_last_error()


def test_workspace_bytes_of_what_no_launch_holds():
    """The query refuses what the calls refuse for its size, and nothing else."""
    none = ctypes.c_size_t(-1).value
    f = mx4._library().indexer_mx4_attend_workspace_bytes
    assert f(2_000_000, 1, 32, 1, 160, 16, 128) == none    # 32 million workgroups of 512 threads
    assert f(2_000_000, 1, 32, 1, 32, 16, 128) == 0        # two heads a wave: 4 million workgroups of 256
    assert f(131072, 1, 32, 1, 64, 64, 192) == 0           # 8.4 million of 256
    assert f(262144, 1, 32, 1, 64, 64, 256) == none        # 16.8 million of 256
    assert f(100_000, 1, 32, 1, 80, 80, 64) == 0
    # prompts of many heads whose keys would be shared out if their join fitted: whole then
    for keys in (1 << 21, 1 << 24, 1 << 30):
        for tokens in (262144, 300_000, 1_000_000):
            for d in (64, 96, 128):
                assert f(1, tokens, keys, 0, 64, 8, d) == 0, (keys, tokens, d)
    # rows of many requests: 512 threads take 256 of a request, or 32 of it
    assert f(5_000_000, 256, 32, 0, 1, 1, 64) == 0
    assert f(9_000_000, 64, 1000, 0, 1, 1, 64) == none


def test_no_call_that_the_query_accepts_is_refused_for_its_size(lib):
    """Random sizes: the query's refusal and the call's are one."""
    rng = np.random.default_rng(7)
    refused = 0
    for _ in range(3000):
        kv = int(rng.choice([1, 2, 8, 16, 64, 128]))
        H = kv * int(rng.integers(1, 1 + min(1024 // kv, 40)))
        d = int(rng.choice([64, 96, 128, 192, 256]))
        Q = int(rng.choice([1, 1, 3, 70, 5000]))
        R = max(1, int(2.0 ** rng.uniform(10, 31)) // (H * Q))
        if R * Q * H > 2**31 - 1024:
            continue
        keys = int(2.0 ** rng.uniform(0, 24))
        selected = int(rng.integers(2))
        need = li.mx4_attend_workspace_bytes(R, Q, keys, bool(selected), H, kv, d)
        shape = dict(R=R, Q=Q, H=H, KV=kv, d=d, qst=H * d, qsh=d, ost=H * d, osh=d, n=keys, idxs=keys, L=keys, bts=keys,
                     bs=1, nb=4, dsb=kv * d // 2, dss=kv * d // 2, dsh=d // 2, ssb=kv * d // 32, sss=kv * d // 32,
                     ssh=d // 32)
        if need == ctypes.c_size_t(-1).value:
            refused += 1
            assert attend(lib, "selected" if selected else "window", **shape) == li.EINVAL
            assert b"too large for one launch" in lib.indexer_last_error()
        elif need:   # a workspace too small is refused after the size: nothing is launched
            assert attend(lib, "selected" if selected else "window", wsn=need - 1, **shape) == li.EWORKSPACE
    assert refused > 20, refused


def test_workspace_bytes_takes_no_size_by_its_low_32_bits():
    need = li.mx4_attend_workspace_bytes(1, 1, 131072, False, 64, 8, 128)
    most = li.mx4_attend_workspace_bytes(1, 1, 2**31 - 1, False, 64, 8, 128)
    assert most >= need > 0
    for keys in (2**31, 2**32 - 2, 2**32 + 32, 2**40):      # window + sinks of the largest windows
        assert li.mx4_attend_workspace_bytes(1, 1, keys, False, 64, 8, 128) == most
    for bad in ((2**32 + 1, 1, 131072, False, 64, 8, 128), (1, 2**32 + 1, 131072, False, 64, 8, 128),
                (1, 1, 131072, False, 2**32 + 64, 8, 128), (1, 1, 131072, False, 64, 8, 2**32 + 128),
                (1, 1, -2**33, False, 64, 8, 128)):
        with pytest.raises(ValueError, match="32-bit"):
            li.mx4_attend_workspace_bytes(*bad)


def test_reading_names_its_own_arguments(lib):
    for kw, msg in ((dict(data=None), b"data is NULL"), (dict(scale=None), b"scale is NULL"),
                    (dict(data=A + 8), b"data must be 16-byte aligned")):
        assert read(lib, **kw) == li.EINVAL
        assert lib.indexer_last_error() == msg
    torch = mx4._torch
    data, scale = torch.zeros((2, 4, 3, 32), dtype=torch.uint8), torch.zeros((2, 4, 3, 2), dtype=torch.uint8)
    dev = data.get_device()
    assert mx4._cache(data, scale, "", dev, 3, 64)[:2] == (2, 4)
    for of in ("", "k_", "v_"):
        with pytest.raises(ValueError, match=f"^{of}scale must be"):
            mx4._cache(data, scale[:1], of, dev, 3, 64)
        with pytest.raises(ValueError, match=f"^{of}data must be"):
            mx4._cache(data, scale, of, dev, 3, 96)
