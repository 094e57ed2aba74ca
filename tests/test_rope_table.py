"""A frequency table that a program copies, as it does when it copies or stores the model that holds it."""
import copy
import ctypes
import pickle

import pytest


@pytest.mark.parametrize("again", [copy.copy, copy.deepcopy, lambda t: pickle.loads(pickle.dumps(t))],
                         ids=["copy", "deepcopy", "pickle"])
def test_copies_have_their_own_frequencies(again):
    import video_dit_block_b200 as sba
    t = sba.rope_frequencies(96, axes=3, scaling="yarn", factor=2.0, original_length=4096)
    want = t.inv_freq, t.axis, t.amplitude, t.rope_dim, t.axes
    c = again(t)
    assert (c.inv_freq, c.axis, c.amplitude, c.rope_dim, c.axes) == want
    # what a call hands over lies in memory that the copy itself keeps
    assert c._freq_at == ctypes.addressof(c._freq) and c._axis_at == ctypes.addressof(c._axis)
    assert tuple(c._freq) == want[0] and tuple(c._axis) == want[1]
