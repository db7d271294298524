"""The forms that calls for requests with a shared prefix take: the sizes of the GPU tests that are meant for one
form take it, so that a changed rule cannot leave a form untested unnoticed."""
import pytest

from mx4_shared_forms import FORMS, kind, of_form, taken


@pytest.mark.parametrize("names", list(FORMS), ids=str)
def test_sizes_take_the_forms_of_their_name(names):
    for d in FORMS[names]:
        assert tuple(kind(f) for f in taken(of_form(names, d))) == names, d


def test_every_form_of_a_part_is_there_at_every_head_dimension():
    """Of the prefix's part and of the own keys', with and without shares."""
    for part, forms in enumerate((("one+", "two", "two+", "prompt", "prompt+", "ahead", "ahead+", "pairs"),
                                  ("one", "one+", "two", "two+", "pairs", "pairs groups", "two groups", "prompt", "ahead"))):
        for name in forms:
            dims = {d for names in FORMS if names[part] == name for d in FORMS[names]}
            narrow = name.startswith(("prompt", "ahead", "pairs", "two groups"))
            assert dims >= ({64, 96, 128} if narrow else {64, 96, 128, 192, 256}), (part, name, dims)
