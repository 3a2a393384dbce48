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


@pytest.mark.parametrize("strings", [[0, 256], [-1, 3], np.array([1.5, 2.0]), np.array([300, 5]), [np.nan, 1], [b"ab"], b"ab"])
def test_strings_that_are_no_bytes_are_refused(strings):
    with pytest.raises(ValueError, match="strings"):
        tt.TokenStrings(strings, [0, 1, 2], device="cpu")


@pytest.mark.parametrize("offsets", [[0, 0.5, 2], [0, np.nan, 2], [0, 1, np.inf]])
def test_offsets_that_are_no_whole_numbers_are_refused(offsets):
    with pytest.raises(ValueError, match="offsets"):
        tt.TokenStrings(np.arange(2), offsets, device="cpu")


def test_strings_of_any_type_that_holds_bytes():
    for strings in (np.arange(256), np.arange(256, dtype=np.uint8), list(range(256)), np.arange(256, dtype=np.int16), np.arange(256.0)):
        assert tt.TokenStrings(strings, [0, 200, 256], device="cpu").strings.tolist() == list(range(256))
    assert tt.TokenStrings([], [0, 0], device="cpu").n_tokens == 1
    assert tt.TokenStrings(np.arange(3), np.array([0.0, 2.0, 3.0]), device="cpu").offsets.tolist() == [0, 2, 3]
