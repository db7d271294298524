"""Sizes that take each form of the 4-bit attention's kernels, and the form a
call takes, so that a test meant for one form can say so (no GPU is needed)."""
import ctypes
from collections import namedtuple

from sparse_attention_lightning_indexer_amd import mx4

# many rows; shared scales; tiles ahead; row tiles and K/V heads of a wave; groups of heads of a
# workgroup; shares of a row's keys; threads of a workgroup
Form = namedtuple("Form", "prompt share ahead tiles heads group splits threads")


def form(requests, query, max_keys, selected, heads, kv, d):
    out = (ctypes.c_int32 * 8)()
    mx4._library().lidx_mx4_attend_form(requests, query, max_keys, int(selected), heads, kv, d, out)
    return Form(*out)


Sizes = namedtuple("Sizes", "lens query heads kv d bs max_seq_len window sinks")


def sizes(lens, query, heads, kv, d, bs, max_seq_len=0, window=50, sinks=3):
    return Sizes(lens, query, heads, kv, d, bs, max_seq_len or max(lens), window, sinks)


FOUR = [60, 33, 5, 70]
LONG = [300, 513, 40, 90] * 4
ROWS = [200, 64, 90, 330] * 4
FORMS = {
    "one tile, 64": sizes([90, 41], 4, 6, 2, 64, 16),
    "one tile, 96": sizes([70, 37], 2, 8, 4, 96, 7),
    "one tile, 128": sizes([70, 37], 4, 8, 2, 128, 16),
    "one tile, 192": sizes([100, 33], 1, 16, 4, 192, 33),
    "one tile, 256": sizes([64, 65], 2, 8, 2, 256, 16),
    "two tiles, 64": sizes([90, 150], 3, 34, 2, 64, 32),
    "two tiles, 96": sizes([90, 150], 3, 34, 2, 96, 32),
    "two tiles, 128": sizes([90, 150], 3, 34, 2, 128, 32),
    "two tiles, 192": sizes([90, 150], 3, 34, 2, 192, 32),
    "two tiles, 256": sizes([90, 150], 3, 34, 2, 256, 32),
    "groups, 64": sizes(FOUR * 16, 8, 32, 8, 64, 16),
    "groups, 96": sizes(FOUR * 16, 8, 32, 8, 96, 16),
    "groups, 128": sizes(FOUR * 16, 8, 32, 8, 128, 16),
    "pairs, 64": sizes(FOUR * 16, 1, 32, 16, 64, 16),
    "pairs, 96": sizes(FOUR * 16, 1, 16, 16, 96, 16),
    "pairs, 128": sizes(FOUR * 16, 1, 64, 16, 128, 16),
    "same keys, 64": sizes(FOUR * 8, 1, 128, 64, 64, 16),
    "same keys, 96": sizes(FOUR * 8, 2, 64, 64, 96, 16),
    "same keys, 128": sizes(FOUR * 8, 1, 128, 64, 128, 16),
    "shared scales, 64": sizes(FOUR * 4, 6, 64, 64, 64, 16),
    "shared scales, 128": sizes(FOUR * 4, 4, 64, 64, 128, 16),
    "shares, 64": sizes([3300, 900], 1, 8, 2, 64, 32, window=1700, sinks=65),
    "shares, 96": sizes([3300, 900], 1, 8, 2, 96, 32, window=1700, sinks=65),
    "shares, 128": sizes([3300, 900], 1, 16, 2, 128, 32, window=1700, sinks=65),
    "shares, 192": sizes([3300, 900], 1, 16, 2, 192, 32, window=1700, sinks=65),
    "shares, 256": sizes([3300, 900], 1, 16, 2, 256, 32, window=1700, sinks=65),
    "two tiles shares, 64": sizes([3300, 900], 1, 40, 2, 64, 32, window=1700, sinks=65),
    "two tiles shares, 96": sizes([3300, 900], 1, 40, 2, 96, 32, window=1700, sinks=65),
    "two tiles shares, 128": sizes([3300, 900], 1, 40, 2, 128, 32, window=1700, sinks=65),
    "two tiles shares, 192": sizes([3300, 900], 1, 40, 2, 192, 32, window=1700, sinks=65),
    "two tiles shares, 256": sizes([3300, 900], 1, 40, 2, 256, 32, window=1700, sinks=65),
    "ahead, 64": sizes(LONG, 1, 16, 16, 64, 16, 2100, 2000, 90),
    "ahead, 96": sizes(LONG, 1, 16, 16, 96, 16, 2100, 2000, 90),
    "ahead, 128": sizes(LONG, 1, 16, 16, 128, 16, 2100, 2000, 90),
    "ahead shares, 64": sizes([4200, 900], 1, 64, 64, 64, 32, window=4095, sinks=5),
    "ahead shares, 96": sizes([4200, 900], 1, 64, 64, 96, 32, window=4095, sinks=5),
    "ahead shares, 128": sizes([4200, 900], 1, 64, 64, 128, 32, window=4095, sinks=5),
    "prompt, 64": sizes(ROWS, 32, 64, 8, 64, 16),
    "prompt, 96": sizes(ROWS, 37, 56, 8, 96, 7),
    "prompt, 128": sizes(ROWS, 64, 32, 8, 128, 64),
    "prompt shares, 64": sizes([4200], 300, 64, 8, 64, 64, window=3500, sinks=30),
    "prompt shares, 96": sizes([4200], 300, 64, 8, 96, 64, window=3500, sinks=30),
    "prompt shares, 128": sizes([4200], 300, 64, 8, 128, 64, window=3500, sinks=30),
}


def max_keys(s, how):
    if how == "selected":
        return min(2048, max(s.lens))
    return s.max_seq_len if how == "causal" else min(s.max_seq_len, s.window + s.sinks)


def taken(name, how):
    s = FORMS[name]
    return form(len(s.lens), s.query, max_keys(s, how), how == "selected", s.heads, s.kv, s.d)


def meant(name):
    """What a form's name says of the form its calls take: {call: {field: value, or a test of it}}."""
    kind = name.split(",")[0]
    many = lambda n: n > 1  # noqa: E731
    plain = dict(prompt=0, share=0, heads=1, group=1, ahead=1)
    every = ("causal", "window", "selected")
    return {
        "one tile": {h: dict(plain, tiles=1, splits=1) for h in every},
        "two tiles": {h: dict(plain, tiles=2, splits=1) for h in every},
        "groups": {h: dict(plain, tiles=2, splits=1, group=many) for h in ("causal", "window")},
        "pairs": {h: dict(plain, tiles=1, splits=1, heads=2) for h in every},
        "same keys": {h: dict(tiles=1, splits=1, heads=2, group=4) for h in every},
        "shared scales": {"selected": dict(share=1, heads=2, group=4)},
        "shares": {h: dict(plain, tiles=1, splits=many) for h in every},
        "two tiles shares": {h: dict(plain, tiles=2, splits=many) for h in every},
        "ahead": {h: dict(plain, tiles=1, splits=1, ahead=2) for h in ("causal", "window")},
        "ahead shares": {h: dict(plain, tiles=1, splits=many, ahead=2) for h in ("causal", "window")},
        "prompt": {h: dict(prompt=1, splits=1) for h in ("causal", "window")},
        "prompt shares": {h: dict(prompt=1, splits=many) for h in ("causal", "window")},
    }[kind]


def agrees(got, want):
    return all(v(getattr(got, k)) if callable(v) else getattr(got, k) == v for k, v in want.items())
