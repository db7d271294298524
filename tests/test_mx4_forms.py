"""The form of the 4-bit attention's kernels that a call takes: the sizes of the GPU tests that are meant for one
form take it, so that a changed rule cannot leave a form untested unnoticed."""
import pytest

from mx4_forms import FORMS, agrees, form, meant, taken


@pytest.mark.parametrize("name", list(FORMS))
def test_sizes_take_the_form_of_their_name(name):
    for how, want in meant(name).items():
        assert agrees(taken(name, how), want), (name, how, taken(name, how), want)


def test_every_head_dimension_of_a_form_is_there():
    dims = {}
    for name, s in FORMS.items():
        dims.setdefault(name.split(",")[0], set()).add(s.d)
    for kind in ("one tile", "two tiles", "shares", "two tiles shares"):
        assert dims[kind] == {64, 96, 128, 192, 256}, kind
    for kind in ("groups", "pairs", "same keys", "ahead", "ahead shares", "prompt", "prompt shares"):
        assert dims[kind] == {64, 96, 128}, kind
    assert dims["shared scales"] == {64, 128}


# sizes of tests in test_mx4_gpu.py: (requests, query, heads, K/V heads, d), then (keys, selected) of its calls

@pytest.mark.parametrize("query,heads,kv,d", [(1, 32, 16, 64), (1, 128, 16, 128), (2, 16, 16, 96), (2, 64, 16, 128)])
def test_pairs_of_heads(query, heads, kv, d):
    for keys, selected in ((70, 1), (63, 1), (149, 0), (43, 0)):
        f = form(64, query, keys, selected, heads, kv, d)
        assert f.heads == 2
        assert f.group == (4 if selected and query == 2 else 1)     # 256 workgroups of 8 heads


@pytest.mark.parametrize("heads,kv,d", [(16, 16, 64), (80, 16, 128), (48, 16, 96)])
def test_two_tiles_ahead(heads, kv, d):
    for keys, selected in ((2100, 0), (2090, 0), (2048, 1), (2304, 1)):
        assert form(16, 1, keys, selected, heads, kv, d).ahead == 2


def test_groups_of_heads():
    for requests, kv, group in ((64, 8, 2), (128, 8, 4), (240, 8, 8), (120, 2, 1)):
        for keys in (89, 35):
            assert form(requests, 8, keys, 0, 4 * kv, kv, 64).group == group


@pytest.mark.parametrize("query,group,d", [(32, 8, 64), (37, 7, 96), (64, 4, 128), (130, 2, 64)])
def test_prompt_rows(query, group, d):
    for keys in (1, 73, 264, 329):
        f = form(16, query, keys, 0, 8 * group, 8, d)
        assert f.prompt and f.splits == 1


def test_prompt_rows_share_keys_out():
    f = form(1, 650, 9000, 0, 16, 8, 64)
    assert f.prompt and f.splits > 1
    assert not form(1, 650, 8030, 0, 16, 8, 64).prompt      # under its window, the wave form
    assert not form(1, 13, 9000, 0, 16, 8, 64).prompt       # the few rows it is compared with


@pytest.mark.parametrize("query,heads,kv,d", [(4, 64, 64, 128), (4, 128, 64, 128), (6, 64, 64, 64), (12, 128, 32, 64)])
def test_shared_scales(query, heads, kv, d):
    for keys in (1, 40, 70, 90, 200, 207):
        assert form(16, query, keys, 1, heads, kv, d).share


@pytest.mark.parametrize("query,heads,kv,d", [(1, 128, 64, 128), (2, 64, 64, 96), (3, 128, 64, 64)])
def test_same_keys_under_a_window(query, heads, kv, d):
    for keys in (1, 37, 64, 110, 128):
        f = form(32, query, keys, 0, heads, kv, d)
        assert f.heads == 2 and f.group == 4 and not f.share


@pytest.mark.parametrize("heads,kv,d", [(3, 1, 64), (20, 2, 96), (5, 1, 192), (40, 2, 256), (17, 1, 256), (4, 4, 128)])
def test_shared_keys(heads, kv, d):
    for keys, selected in ((3300, 0), (1765, 0), (2000, 1), (1920, 1)):
        assert form(2, 1, keys, selected, heads, kv, d).splits > 1
