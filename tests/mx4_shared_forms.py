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


def kind(form):
    """A form in a word; "+" where a row's keys are in shares."""
    if form.splits == 0:
        return "none"
    word = "prompt" if form.prompt else "pairs" if form.heads == 2 else "two" if form.tiles == 2 else (
        "ahead" if form.ahead == 2 else "one")
    return word + (" groups" if form.group > 1 else "") + ("+" if form.splits > 1 else "")


def sizes(requests, query, prefix, own, groups, heads, kv, d, bs=16):
    """Groups of one size (the last smaller), prefixes up to `prefix`, own keys up to `own`; a request of none among them."""
    most = -(-requests // groups)
    starts = [min(g * most, requests) for g in range(groups + 1)]
    owns = [max(query, own - (7 * r) % max(1, own // 2)) for r in range(requests)]
    if requests > 3:
        owns[2] = 0
    prefixes = [prefix - (5 * g) % max(1, prefix // 3) for g in range(groups)]
    return Sizes(starts, prefixes, owns, query, heads, kv, d, bs)


# (form of the prefix's part, form of the own keys'): sizes that take them, of every head dimension they have
FORMS = {
    ("none", "one"): {64: (2, 1, 64, 8, 1, 1, 1), 96: (2, 4, 64, 8, 1, 1, 1), 128: (3, 2, 64, 8, 1, 1, 1),
                      192: (3, 4, 64, 8, 1, 1, 1), 256: (3, 1, 64, 8, 1, 1, 1)},
    ("none", "one+"): {64: (2, 1, 3000, 8, 1, 1, 1), 96: (2, 1, 1500, 600, 1, 1, 1), 128: (3, 1, 1500, 8, 1, 1, 1),
                       192: (2, 1, 400, 200, 1, 1, 1), 256: (2, 4, 400, 200, 1, 1, 1)},
    ("none", "ahead"): {64: (128, 1, 3000, 8, 1, 2, 2), 96: (200, 2, 3000, 8, 1, 1, 1), 128: (200, 4, 3000, 8, 1, 1, 1)},
    ("none", "ahead+"): {64: (48, 4, 12000, 8, 1, 1, 1), 96: (48, 4, 12000, 200, 1, 4, 1), 128: (100, 4, 6000, 8, 8, 4, 1)},
    ("none", "pairs"): {64: (128, 4, 64, 8, 1, 8, 8), 96: (64, 2, 64, 8, 1, 16, 16), 128: (128, 4, 64, 8, 1, 8, 8)},
    ("none", "pairs groups"): {64: (128, 1, 64, 8, 1, 16, 16), 96: (128, 2, 64, 8, 1, 16, 16),
                               128: (128, 1, 64, 8, 2, 64, 16)},
    ("none", "two"): {64: (2, 32, 64, 64, 1, 1, 1), 96: (3, 32, 64, 32, 1, 1, 1), 128: (3, 32, 64, 32, 1, 1, 1),
                      192: (2, 32, 64, 64, 1, 1, 1), 256: (2, 32, 64, 64, 1, 1, 1)},
    ("none", "two+"): {64: (3, 100, 1500, 100, 1, 1, 1), 96: (3, 32, 1500, 32, 1, 1, 1), 128: (2, 32, 1500, 32, 1, 1, 1),
                       192: (3, 100, 400, 200, 1, 1, 1), 256: (2, 100, 400, 200, 1, 1, 1)},
    ("none", "two groups"): {64: (64, 4, 64, 8, 1, 64, 8), 96: (64, 100, 400, 100, 1, 2, 2), 128: (64, 32, 200, 32, 8, 8, 2)},
    ("none", "prompt"): {64: (24, 100, 64, 100, 1, 4, 1), 96: (48, 32, 64, 32, 1, 8, 1), 128: (200, 4, 64, 8, 1, 16, 1)},
    ("none", "prompt+"): {64: (100, 100, 1500, 100, 8, 2, 1), 96: (100, 100, 3000, 100, 2, 2, 1),
                          128: (128, 100, 1500, 100, 1, 2, 1)},
    ("one", "pairs groups"): {64: (128, 1, 800, 64, 8, 16, 16), 96: (128, 1, 400, 8, 8, 16, 16), 128: (64, 1, 400, 8, 8, 32, 32)},
    ("one", "one"): {128: (100, 1, 800, 64, 8, 8, 8), 192: (64, 1, 800, 8, 8, 32, 16), 256: (64, 1, 200, 8, 8, 32, 32)},
    ("one+", "one"): {64: (128, 1, 6000, 64, 8, 1, 1), 96: (100, 1, 6000, 8, 8, 1, 1), 128: (100, 1, 3000, 8, 8, 1, 1),
                      192: (100, 1, 1500, 64, 8, 1, 1), 256: (100, 1, 3000, 8, 8, 1, 1)},
    ("one+", "pairs"): {64: (128, 1, 1500, 64, 8, 8, 8), 96: (128, 1, 3000, 8, 8, 8, 8), 128: (128, 1, 1500, 8, 8, 8, 8)},
    ("one+", "one+"): {192: (100, 1, 6000, 1500, 8, 1, 1)},
    ("two", "one"): {64: (100, 4, 3000, 64, 1, 16, 8), 96: (200, 4, 3000, 8, 1, 8, 4), 128: (200, 4, 1500, 64, 1, 8, 4),
                     192: (200, 4, 400, 8, 1, 16, 16), 256: (200, 4, 800, 8, 1, 8, 8)},
    ("two", "pairs"): {64: (200, 4, 1500, 8, 1, 8, 8), 96: (200, 4, 800, 8, 1, 8, 8), 128: (200, 4, 800, 8, 1, 8, 8)},
    ("two+", "one"): {64: (200, 1, 6000, 8, 1, 1, 1), 96: (100, 1, 6000, 8, 1, 1, 1), 128: (200, 1, 3000, 8, 1, 1, 1),
                      192: (200, 1, 1500, 8, 1, 1, 1), 256: (128, 4, 3000, 8, 1, 1, 1)},
    ("two+", "pairs groups"): {64: (128, 1, 800, 8, 1, 16, 16), 96: (200, 1, 400, 8, 1, 16, 16), 128: (128, 2, 400, 8, 1, 16, 16)},
    ("two+", "two"): {64: (24, 100, 12000, 100, 1, 1, 1), 96: (24, 100, 6000, 200, 1, 1, 1), 128: (24, 100, 6000, 200, 1, 1, 1),
                      192: (48, 100, 1500, 100, 1, 1, 1), 256: (24, 100, 1500, 100, 1, 1, 1)},
    ("two+", "two+"): {128: (24, 100, 12000, 3000, 1, 1, 1), 192: (12, 100, 12000, 600, 1, 1, 1), 256: (12, 100, 6000, 1500, 1, 2, 2)},
    ("two+", "one+"): {96: (100, 1, 12000, 3000, 1, 1, 1), 192: (48, 2, 12000, 600, 1, 1, 1), 256: (48, 1, 12000, 600, 1, 1, 1)},
    ("prompt", "one"): {64: (200, 4, 1500, 8, 2, 64, 16), 96: (128, 4, 800, 8, 1, 128, 32), 128: (200, 4, 1500, 8, 1, 64, 16)},
    ("prompt", "prompt"): {64: (64, 100, 12000, 100, 2, 8, 8), 96: (64, 100, 6000, 200, 1, 8, 8),
                           128: (128, 100, 6000, 100, 1, 4, 4)},
    ("prompt+", "one"): {64: (200, 4, 12000, 200, 1, 4, 2), 96: (200, 4, 12000, 8, 1, 4, 2), 128: (200, 4, 3000, 8, 1, 16, 4)},
    ("prompt+", "two groups"): {64: (32, 32, 3000, 1500, 1, 16, 2), 96: (128, 32, 6000, 32, 1, 8, 8),
                                128: (64, 100, 6000, 200, 1, 2, 2)},
    ("prompt+", "ahead"): {64: (128, 4, 12000, 3000, 1, 8, 2), 128: (200, 2, 12000, 3000, 1, 8, 1)},
    ("prompt+", "prompt"): {64: (200, 100, 6000, 100, 1, 8, 1), 96: (100, 100, 6000, 100, 1, 2, 1),
                            128: (100, 100, 6000, 100, 1, 2, 1)},
    ("prompt+", "prompt+"): {96: (100, 100, 12000, 1500, 1, 2, 1)},
    ("ahead", "one"): {64: (128, 1, 3000, 8, 64, 4, 4), 96: (128, 1, 3000, 8, 64, 4, 4), 128: (100, 1, 3000, 64, 50, 4, 4)},
    ("ahead+", "one"): {64: (100, 2, 12000, 200, 50, 1, 1), 96: (200, 1, 6000, 8, 100, 1, 1), 128: (200, 1, 6000, 8, 100, 1, 1)},
    ("pairs", "pairs groups"): {64: (128, 2, 800, 8, 64, 16, 16), 96: (200, 2, 400, 8, 100, 16, 16),
                                128: (200, 2, 400, 8, 100, 16, 16)},
}


def of_form(names, d):
    return sizes(*FORMS[names][d], d)
