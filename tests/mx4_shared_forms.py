"""Sizes that take each form of the attention of requests that share a prefix,
and the forms its two parts take (no GPU is needed)."""
import ctypes
from collections import namedtuple

from mx4_forms import Form
from sparse_attention_lightning_indexer_amd import mx4

# starts and prefixes of the groups, each request's own keys behind the prefix
Sizes = namedtuple("Sizes", "starts prefixes own query heads kv d bs")


def forms(requests, query, max_seq_len, groups, max_group, max_prefix, heads, kv, d):
    """The forms of the prefix's part and of the requests' own."""
    sizes = (ctypes.c_int32 * 9)(requests, query, max_seq_len, groups, max_group, max_prefix, heads, kv, d)
    out = (ctypes.c_int32 * 16)()
    mx4._library().lidx_mx4_shared_form(sizes, out)
    return Form(*out[:8]), Form(*out[8:])


def lens(s):
    out = [0] * len(s.own)
    for r, own in enumerate(s.own):
        group = [g for g in range(len(s.prefixes)) if s.starts[g] <= r < s.starts[g + 1]]
        out[r] = own + (s.prefixes[group[0]] if group and own else 0)
    return out


def taken(s):
    count = max(b - a for a, b in zip(s.starts, s.starts[1:]))
    return forms(len(s.own), s.query, max(lens(s)), len(s.prefixes), count, max(s.prefixes), s.heads, s.kv, s.d)
