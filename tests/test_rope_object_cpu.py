"""A Rope as part of a module: copied, saved, sent to another process, and not changed behind the library's back."""
import copy
import ctypes
import pickle

import pytest

from mxfp4_precision_gemms_gb300 import binding as mx


def _read(rope):
    """What the library reads: the frequencies, the axes, pairs, interleaved."""
    c = mx.RopeC.from_address(rope.ref)
    axis = c.axis and list((ctypes.c_int32 * c.pairs).from_address(c.axis))
    return list((ctypes.c_double * c.pairs).from_address(c.freq)), axis, c.pairs, c.interleaved


@pytest.mark.parametrize("rope", [mx.Rope([1.0, 0.5, 0.25]), mx.Rope([1.0, 1e-3], axis=[2, 0], interleaved=True)])
def test_copies(rope):
    import io

    import torch

    file = io.BytesIO()
    torch.save({"rope": rope}, file)
    file.seek(0)
    want = _read(rope)
    for made in (copy.copy(rope), copy.deepcopy(rope), pickle.loads(pickle.dumps(rope)),
                 torch.load(file, weights_only=False)["rope"]):
        assert made is not rope and made.ref != rope.ref and _read(made) == want
        assert (made.axes, made.interleaved) == (rope.axes, rope.interleaved)


def test_a_module_that_holds_one():
    import torch

    class Block(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.rope, self.gain = mx.Rope([1.0, 0.5]), torch.nn.Parameter(torch.ones(4))

    block = Block()
    other = copy.deepcopy(block)
    del block
    assert _read(other.rope) == ([1.0, 0.5], None, 2, 0)


def test_its_arrays_stay_where_they_are():
    """The library reads them at their addresses: they take new numbers, but no other length."""
    rope = mx.Rope([1.0, 0.5], axis=[0, 1])
    for change in (lambda: rope.freq.extend([0.0] * 100000), lambda: rope.axis.append(0), lambda: rope.freq.pop()):
        with pytest.raises(BufferError):
            change()
    rope.freq[1] = 0.25
    assert _read(rope) == ([1.0, 0.25], [0, 1], 2, 0)
