"""Grammars and token strings keep the tensors that their addresses stand for; copies have their own (no GPU needed)."""
import copy
import gc
import pickle
import struct
import weakref

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import exact_byte_level_amd as tt  # noqa: E402


def made():
    nxt = np.full((3, 256), -1)
    nxt[0, 97:123] = 1
    return [(tt.Grammar(nxt, device="cpu"), ("classes", "next", "accept"), (0, 1, 2)),
            (tt.TokenStrings(np.arange(9), [0, 1, 5, 9], device="cpu"), ("strings", "offsets"), (0, 2))]


@pytest.mark.parametrize("which", [0, 1])
def test_a_tensor_that_is_replaced_stays_alive(which):
    handle, names, _ = made()[which]
    fields = handle._fields
    for name in names:
        old = weakref.ref(getattr(handle, name))
        setattr(handle, name, None)
        gc.collect()
        assert old() is not None
    assert handle._fields == fields


@pytest.mark.parametrize("again", [copy.copy, copy.deepcopy, lambda h: pickle.loads(pickle.dumps(h))], ids=["copy", "deepcopy", "pickle"])
@pytest.mark.parametrize("which", [0, 1])
def test_a_copy_points_to_its_own_tensors(which, again):
    handle, names, places = made()[which]
    other = again(handle)
    fields = struct.unpack("=%dq" % (len(other._fields) // 8), other._fields)
    assert [fields[p] for p in places] == [getattr(other, n).data_ptr() for n in names]
    assert all(torch.equal(getattr(other, n), getattr(handle, n)) for n in names)
    rest = [i for i in range(len(fields)) if i not in places]
    before = struct.unpack("=%dq" % len(fields), handle._fields)
    assert [fields[i] for i in rest] == [before[i] for i in rest]
