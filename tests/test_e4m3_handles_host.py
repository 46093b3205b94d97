"""Handles of 8-bit rows and weights without a GPU."""
import pytest
import torch

from test_e4m3_host import SCALE, codes, on_gpu, rows, weight  # noqa: F401 (on_gpu is a fixture)


@pytest.mark.parametrize("make", [rows, weight])
def test_a_handle_keeps_what_it_was_made_of(on_gpu, make):  # noqa: F811
    """The calls take the pointers and counts read at the start: another tensor in a
    handle's attribute would be ignored, and the one that they use be freed."""
    x = make(256, 144)
    was = (x.codes, x.scale, x._struct.codes, x._struct.scale)
    for name, value in (("codes", codes(256, 144)), ("scale", codes(256, 2, dtype=SCALE)), ("rows", 3), ("cols", 16), ("dev", 1),
                        ("_struct", None), ("_ref", None), ("other", 1)):
        with pytest.raises(AttributeError, match=name):
            setattr(x, name, value)
    for name in ("codes", "scale", "rows"):
        with pytest.raises(AttributeError, match=name):
            delattr(x, name)
    assert (x._struct.codes, x._struct.scale) == was[2:]
    assert x.codes is was[0] and x.scale is was[1] and (x.rows, x.cols, x.dev) == (256, 144, 0)
    assert x.codes.data_ptr() == x._struct.codes and x.scale.data_ptr() == x._struct.scale
    x.codes.view(torch.uint8).fill_(1)                 # what they hold may change
